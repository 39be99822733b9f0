"""The bounds-checked build on the chunk, rotary and append tests, and what surrounds a given workspace.

In ``libbfa_checked.so`` the page look-ups, rows of q and out, cuts and workspace places of these kernels
check their bounds; an index outside its array is skipped and reported by ``chunk_device_status``, which
the plugin asks after every test.
"""

import os
import subprocess
import sys

import pytest
import torch

from test_gpu_chunk import Batch, bfa

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

CASES = ["test_gpu_chunk.py::" + n for n in (
    "test_single_tokens", "test_head_layouts", "test_chunks_of_all_lengths", "test_lengths_around_the_tiles",
    "test_rows_behind_the_last_sequence_stay", "test_long_context_is_cut_into_pieces",
    "test_pages_that_do_not_exist_read_as_zeros", "test_lengths_beyond_the_table_count_as_its_room",
    "test_strides_scale_and_given_results", "test_many_sequences", "test_empty_calls",
    "test_a_given_workspace_with_anything_in_it")] + ["test_gpu_rope.py::" + n for n in (
        "test_rope", "test_rope_forms_of_the_arguments", "test_append",
        "test_append_leaves_out_places_that_do_not_exist", "test_serving_in_steps_equals_the_whole_prompt")]


def test_the_checked_build_finds_no_index_out_of_bounds():
    if os.environ.get("BFA_LIBRARY") == "checked":
        pytest.skip("already the checked build")
    env = dict(os.environ, BFA_LIBRARY="checked", PYTHONPATH=os.pathsep.join([HERE, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu", "-p", "no:cacheprovider", "-p",
                        "checked_chunk_status"] + ["tests/" + n for n in CASES],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:] + r.stderr[-1000:]


@pytest.mark.parametrize("q_lens,kv", [([1] * 9, [5000, 3, 700, 0, 64, 9000, 128, 1, 2500]), ([300, 1, 40], [5000, 900, 300]),
                                       ([2000], [9000])])
def test_nothing_around_the_workspace_is_written(q_lens, kv):
    b = Batch(q_lens, kv, 8, 2, 128, 16)
    want = b.call()
    need = bfa._L.bfa_fwd_chunk_workspace(sum(q_lens), len(q_lens), max(q_lens), 8, 2, 128)
    room = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    got = b.call(workspace=room[4096:4096 + need])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (room[:4096] == 0xA5).all() and (room[4096 + need:] == 0xA5).all()
