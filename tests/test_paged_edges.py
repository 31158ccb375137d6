"""Paged-cache and beam operators at the edges of what they take: what a CPU can check."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def source(name):
    return open(os.path.join(ROOT, "confidence_gated_kv_logits_gb300", "csrc", name)).read()


def test_softmax_warps_leave_their_loop_together():
    """Barriers of some of a block's warps wait without a limit, so after a wait that gave up (2 s) no warp may leave the
    others at one: the loop over pieces ends by a decision of all warps, and nothing that can give up lies between the
    second of its decisions and the next turn."""
    role = source("k_paged_attend_many.cu").split("// ---- softmax and epilogue ----")[1].split("\ntemplate ")[0]
    loop = re.search(r"\n    while \((.*)\) \{\n", role)
    assert loop.group(1) == "!soft_any(!next_piece())"
    body = role[loop.end():role.index("\n    }\n", loop.end())]
    leave = re.findall(r"\n      (.*(?:break|return);.*)", "\n".join(x for x in body.split("\n") if re.match(r"      \S", x)).join("\n\n"))
    assert len(leave) == 1 and leave[0].startswith("if (soft_any(")
    before, after = body.split(leave[0])
    assert "bar_wait" in before and "soft_sync" not in before
    assert "bar_wait" not in after and "next_piece" not in after


# --------------------------------------------------------------------------- the binding
@pytest.fixture(scope="module")
def pkg():
    from confidence_gated_kv_logits_gb300 import build as B
    B.build()
    import confidence_gated_kv_logits_gb300 as pkg
    from confidence_gated_kv_logits_gb300.paged import _load
    _load()
    return pkg


def test_a_scale_that_is_zero_in_32_bits_is_refused(pkg):
    """It would mean the default."""
    import torch
    from confidence_gated_kv_logits_gb300 import _paged_ops as ops
    ob = ops.make(4096, 0, 0, 0, 2, 1, 64, 0, -1, 0)
    # (the tensors are on the CPU: any other scale is refused for that)
    with pytest.raises(ValueError, match="q: want"):
        ops.attend(ob, 0, -1, 0, torch.zeros(1, 2, 64).half(), torch.zeros(1, 2, 64).half(), None, 1.0, None)
    with pytest.raises(ValueError, match="scale"):
        ops.attend(ob, 0, -1, 0, torch.zeros(1, 2, 64).half(), torch.zeros(1, 2, 64).half(), None, 1e-60, None)
    ops.release(ob)


def test_a_closed_handle_says_so(pkg):
    """Every call, status without its check among them (which answered 0: no flags)."""
    from confidence_gated_kv_logits_gb300.paged import BatchStruct, PagedBatch
    kv = pkg.PagedKV.__new__(pkg.PagedKV)
    kv._L, kv._h, kv._ob, kv._index = pkg.load_library(), None, None, 0
    batch = PagedBatch(BatchStruct(), (), 1, -1, 0)
    for call in (lambda: kv.append(0, batch, None, None), lambda: kv.attend(0, batch, None, None), lambda: kv.commit(*[None] * 5),
                 lambda: kv.fork(*[None] * 7), lambda: kv.status(), lambda: kv.status(check=False)):
        with pytest.raises(ValueError, match="closed"):
            call()
    kv.close()


def test_beam_select_on_the_device_that_was_named(pkg, monkeypatch):
    import torch
    from confidence_gated_kv_logits_gb300 import paged
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)

    def scratch(self, n, zeroed):
        self._home = 0
        return 4096

    monkeypatch.setattr(paged.BeamSelect, "_scratch", scratch)
    for device, index in ((None, 3), ("cuda", 3), (torch.device("cuda"), 3), ("cuda:1", 1), (torch.device("cuda", 0), 0), (2, 2), (0, 0)):
        assert pkg.BeamSelect(1, 2, 100, 4, device=device).device == torch.device("cuda", index)
    for device in ("cpu", torch.device("meta")):
        with pytest.raises(ValueError, match="CUDA"):
            pkg.BeamSelect(1, 2, 100, 4, device=device)


# --------------------------------------------------------------------------- the build
@pytest.fixture
def builder(monkeypatch, tmp_path):
    """The build with its objects in place and its two results elsewhere; `ran` gets the commands that it runs."""
    from confidence_gated_kv_logits_gb300 import build as B
    B.build()
    B.ran = []
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libconfkv.so"))
    monkeypatch.setattr(B, "OPS", str(tmp_path / "_paged_ops.so"))

    def link_library(cmd, **kw):
        B.ran.append("library")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return type("Done", (), {"returncode": 0, "stderr": ""})

    monkeypatch.setattr(B.subprocess, "run", link_library)
    monkeypatch.setattr(B, "_run", lambda cmd, what: (B.ran.append("module"), open(cmd[cmd.index("-o") + 1], "w").close()))
    return B


def test_the_library_is_built_without_torch(builder, monkeypatch):
    monkeypatch.setattr(builder.importlib.util, "find_spec", lambda name: None)
    assert os.path.exists(builder.build()) and builder.ran == ["library"]
    assert not os.path.exists(builder.OPS)


def test_the_library_is_linked_where_the_module_does_not_compile(builder, monkeypatch):
    def broken(*a):
        raise RuntimeError("g++ found no Python.h")

    monkeypatch.setattr(builder, "_ops_object", broken)
    monkeypatch.setattr(builder, "_ops_stale", lambda *a: True, raising=False)
    monkeypatch.setattr(builder, "_stale", lambda target, deps: not os.path.exists(target) or target.endswith("paged_py.o"))
    with pytest.raises(RuntimeError, match="Python.h"):
        builder.build()
    assert os.path.exists(builder.LIB) and not os.path.exists(builder.OPS)


def test_the_module_is_built_anew_for_another_torch(builder, monkeypatch, tmp_path):
    torch = builder._torch()
    src, obj = str(tmp_path / "a.cpp"), str(tmp_path / "a.o")
    open(src, "w").close()
    builder._ops_object(src, obj, torch)
    assert builder.ran == ["module"] and not builder._ops_stale(src, obj, [], torch)
    other = tmp_path / "torch"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '0'")
    assert builder._ops_stale(src, obj, [], str(other))
