"""pytest plugin for runs of the bounds-checked library: after each test, the status word that the chunk,
rotary and append kernels share must hold no index error."""

import pytest


@pytest.fixture(autouse=True)
def _chunk_status():
    import mask_skipping_flashattention_b200 as bfa

    yield
    bfa.chunk_device_status()
