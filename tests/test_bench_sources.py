"""The hash that ties the committed profiles to the kernels they were taken on."""

import os
import shutil

import bench


def test_hash_follows_the_forward_kernels_only(tmp_path, monkeypatch):
    csrc = os.path.join("free_ffn_activation_prox_amd", "csrc")
    shutil.copytree(os.path.join(bench.ROOT, csrc), tmp_path / csrc)
    shutil.copytree(os.path.join(bench.ROOT, "include"), tmp_path / "include")
    here = bench.kernel_sources_hash()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_sources_hash() == here

    def touched(name):
        path = tmp_path / csrc / name
        text = path.read_text()
        path.write_text(text + "// more\n")
        changed = bench.kernel_sources_hash() != here
        path.write_text(text)
        return changed

    for name in ("prox_kv.hip", "prox_kv.hpp", "prox_kv_api.hip", "prox_kv_attn.hip"):
        assert not touched(name), name
    for name in ("prox_kernels.hip", "prox_batch.hip", "prox_device.hpp", "prox_internal.hpp"):
        assert touched(name), name
