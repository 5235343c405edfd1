"""The serving operators' extension module: the rest of the package works without it."""
import os
import subprocess
import sys

import pytest

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-3000:]
    return out.stdout


def test_the_package_works_without_it():
    """Inference and training keep to ctypes; a serving operator says what is missing when it is called."""
    said = run("""
import sys
sys.modules["hashed_gram_memory_tid2eid_amd._tensor_args"] = None  # cannot be imported
import torch
import hashed_gram_memory_tid2eid_amd as eng
assert eng.engram_build_id() and eng.Engram and eng.SiteTraining
eng.engram_layout_create(vocab_size=100, compressed_vocab=50, pad_token_id=0, heads_per_order=1, rows=[1000] * 3, row_dim=64,
                         table_dtype=eng.ENGRAM_DTYPE_BF16, row_pitch_bytes=128)
assert eng.engram_embed_grad_workspace(100, 1000, 64) > 0
assert eng.engram_beam_select_workspace(1, 4, 1000, 4) > 0
t = torch.zeros((2, 3), dtype=torch.int32)
for call in (lambda: eng.engram_state_copy(t, t[0], t[0]), lambda: eng.engram_beam_reorder(t, slots=t),
             lambda: eng.engram_block_release(t, t, t, t, page_size=1, num_pages=1),
             lambda: eng.engram_beam_select(t, t, t, t, t, workspace=t),
             lambda: eng.engram_block_plan(t, t, t, t, page_size=1, num_pages=1, cu_seqlens=t, token_slots=t)):
    try:
        call()
    except ImportError as e:
        print(e)
""")
    assert said.count("build_lib.py") == 5


def build_lib():
    import runpy
    return runpy.run_path(os.path.join(ROOT, "hashed_gram_memory_tid2eid_amd", "build_lib.py"))


def test_it_records_what_it_was_built_for(monkeypatch):
    """Its source, its flags, the torch and the Python: another of these and it is built again."""
    import torch
    bl = build_lib()
    identity, built, ensure = bl["tensor_args_identity"], bl["built_tensor_args"], bl["ensure_built"]
    now = identity()
    assert built() == now and built(os.path.join(ROOT, "README.md")) is None and built("/nowhere") is None
    asked = []
    monkeypatch.setitem(ensure.__globals__, "build", lambda: asked.append(1) or "built")
    assert ensure() == bl["LIB"] and not asked
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        assert identity() != now and ensure() == "built"
    with monkeypatch.context() as m:
        m.setitem(identity.__globals__, "EXT_SUFFIX", ".cpython-399-x86_64-linux-gnu.so")
        assert identity() != now and ensure() == "built"
    with monkeypatch.context() as m:
        m.setitem(identity.__globals__, "TENSOR_ARGS_FLAGS", bl["TENSOR_ARGS_FLAGS"] + ["-O3"])
        assert identity() != now and ensure() == "built"
    assert identity() == now and len(asked) == 3
    # no other Python takes it for its own
    assert bl["TENSOR_ARGS"].endswith(bl["EXT_SUFFIX"]) and "cpython-" in bl["EXT_SUFFIX"]


def test_it_is_not_used_with_another_torch():
    said = run("""
import torch
torch.__version__ = "0.0.1"
import hashed_gram_memory_tid2eid_amd as eng
t = torch.zeros((2, 3), dtype=torch.int32)
try:
    eng.engram_state_copy(t, t[0], t[0])
except ImportError as e:
    print(e, "|", e.__cause__)
""")
    assert "build_lib.py" in said and "0.0.1" in said
