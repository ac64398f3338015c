"""The C++ half of the Python binding is a short way to calls that ctypes makes as
well: a program without it (only libkd.so was built, or the module is of another torch)
keeps every entry point.  And a module that was built for another torch or Python is built
again."""

import subprocess
import sys
import textwrap

import pytest

from chunked_kl_loss_chunk_b200 import build, kd

ROOT = build.ROOT


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kd.load()


def test_every_call_without_the_module():
    """In a process where the module cannot be imported."""
    code = textwrap.dedent("""
        import sys, warnings
        class Absent:
            def find_spec(self, name, path=None, target=None):
                if name.endswith("_kd_native"):
                    raise ImportError("no such module here")
        sys.meta_path.insert(0, Absent())
        import torch
        from chunked_kl_loss_chunk_b200 import kd
        with warnings.catch_warnings(record=True) as seen:
            warnings.simplefilter("always")
            assert kd.load() is kd.load()
        assert len(seen) == 1 and "_kd_native" in str(seen[0].message), seen
        assert kd.load().kd_version() >> 16 == 1
        assert kd.kd_fused_kl_fwd(None, None, 1, 4, 8, 8, None, None, 1, 4, 1.0, None, None, None, None, 0, None) \
            == kd.KD_ERR_INVALID_ARG
        x, a, i = torch.zeros(4, 8), torch.zeros(4), torch.zeros(4, dtype=torch.int32)
        for call in (lambda: kd.policy_loss(x, x, a), lambda: kd.preference_loss(x), lambda: kd.clip_grad_norm([x], 1.0),
                     lambda: kd.head_logprobs(x, x, i, 4), lambda: kd.head_logprobs_bwd(x, x, i, a, a, 4)):
            try:
                call()
            except ValueError as e:           # kd.py's own checks: these tensors are on the CPU
                assert "CUDA" in str(e), e
            else:
                raise AssertionError("not refused")
        print("fine")
    """)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stdout + r.stderr


def test_the_library_alone_can_be_built(monkeypatch):
    """No compiler for the module, no torch headers: libkd.so is there all the same."""
    def no_module(*a, **k):
        raise AssertionError("the module was asked for")
    monkeypatch.setattr(build, "build_native", no_module)
    assert build.build(native=False) == build.LIB_PATH


def test_a_module_of_another_torch_is_built_again(monkeypatch, tmp_path):
    ran = []

    def compiler(cmd, check):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "NATIVE_PATH", str(tmp_path / "_kd_native.so"))
    monkeypatch.setattr(build, "NATIVE_STAMP", str(tmp_path / "stamp"))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    build.build_native()
    build.build_native()
    assert len(ran) == 1                       # up to date
    import torch
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    build.build_native()
    build.build_native()
    assert len(ran) == 2
    monkeypatch.setattr(build.sys, "version_info", (9, 9, 9, "final", 0))
    build.build_native()
    assert len(ran) == 3
    (tmp_path / "stamp").unlink()              # made by an older build.py
    build.build_native()
    assert len(ran) == 4
