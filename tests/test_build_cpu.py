"""When the extension module is built again: sources, torch, Python and C++ ABI."""

import os

from rope_context_extension_scaled_b200 import build


def test_extension_built_against_another_torch_is_out_of_date(tmp_path, monkeypatch):
    so, abi = tmp_path / "_rcx_torch.so", tmp_path / "_rcx_torch.abi"
    monkeypatch.setattr(build, "EXT", str(so))
    monkeypatch.setattr(build, "EXT_ABI", str(abi))
    assert not build.ext_up_to_date()                          # not built
    so.write_bytes(b"")
    assert not build.ext_up_to_date()                          # built by who knows what
    abi.write_text(build.ext_abi())
    assert build.ext_up_to_date()
    for other in (build.ext_abi().replace("torch ", "torch 0"), build.ext_abi().replace("python ", "python 0"), ""):
        abi.write_text(other)
        assert not build.ext_up_to_date()
    abi.write_text(build.ext_abi())
    os.utime(so, (0, 0))                                       # older than its sources
    assert not build.ext_up_to_date()
