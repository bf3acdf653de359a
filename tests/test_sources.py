"""What the CUDA sources leave out."""
import pathlib
import re

ROOT = pathlib.Path(__file__).resolve().parent.parent


def test_no_load_is_multicast():
    """A bulk load names one CTA: the library also runs in processes of several GPUs (the sharded lookup), where
    loads that write into several CTAs' shared memory have no place."""
    for path in sorted((ROOT / "gram_hash_embedding_gb300" / "csrc").iterdir()) + sorted((ROOT / "synth").glob("*.cu")):
        for line in path.read_text().splitlines():
            assert not (re.search(r"cp\.async\.bulk", line) and "multicast" in line), f"{path.name}: {line.strip()}"
