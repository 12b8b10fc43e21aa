"""The binding and the build of the decoder-block operators on the CPU: what is refused before any launch."""
import os
import shutil
import subprocess

import pytest
import torch

import block_quantized_routed_gb300 as moe
from block_quantized_routed_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()
    moe.load()


def calls():
    """Each operator with tensors that are right but for their device."""
    x, w = torch.zeros(2, 256), torch.ones(256)
    yield "norm", lambda: moe.moe_add_rmsnorm(x, w, 1e-6, residual=x, sum_out=x, y=x.clone(), q_fmt=moe.NORM_Q_Q8K,
                                              q=torch.zeros(2, 256, dtype=torch.int8), d=torch.zeros(2, 1),
                                              bsum16=torch.zeros(2, 16, dtype=torch.int16))
    yield "route", lambda: moe.moe_route_grouped(x, 4, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4),
                                                 bias=torch.zeros(256))
    kc = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    table, cu = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    n, kn = torch.zeros(2, dtype=torch.int32), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    ws = torch.zeros(moe.moe_paged_attention_workspace_size(4, 2, 64), dtype=torch.uint8)
    yield "append", lambda: moe.moe_kv_append(kn, kn, kc, kc, table, cu, n, ws)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    yield "attention", lambda: moe.moe_paged_attention(q, kc, kc, table, cu, n, 0.1, torch.empty_like(q), ws,
                                                       lse=torch.zeros(3, 4))


@pytest.mark.parametrize("name", ["norm", "route", "append", "attention"])
def test_tensors_of_the_host_are_refused(name):
    """A tensor that is right in every other way: its pointer would reach a kernel."""
    with pytest.raises(moe.MoeError) as e:
        dict(calls())[name]()
    assert e.value.status == moe.MOE_ERR_INVALID_ARG and "GPU" in str(e.value)


def test_workspaces_have_to_be_contiguous():
    """An expanded workspace has fewer bytes than elements."""
    kc = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    table, cu, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1, dtype=torch.uint8).expand(1 << 20)
    with pytest.raises(moe.MoeError, match="contiguous"):
        moe.moe_kv_append(q[:, :2], q[:, 2:], kc, kc, table, cu, n, ws)
    with pytest.raises(moe.MoeError, match="contiguous"):
        moe.moe_paged_attention(q, kc, kc, table, cu, n, 0.1, torch.empty_like(q), ws)


def test_a_flag_without_a_truth_value_is_an_error():
    x = torch.zeros(2, 256)
    with pytest.raises(RuntimeError, match="ambiguous|Boolean"):
        moe.moe_route_grouped(x, 4, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4), renorm=torch.ones(2))


PER_DEVICE = r"""
#include <cassert>
#include <thread>
#include <vector>
#include "moe_per_device.h"
static thread_local int current = 0;
extern "C" cudaError_t cudaGetDevice(int* dev) { *dev = current; return cudaSuccess; }
int main() {
  moe::PerDevice kept;
  int asked = 0;
  const auto get = [&](int dev) { ++asked; return 100 + dev; };
  assert(kept(get) == 100 && kept(get) == 100 && asked == 1);
  current = 1;                                              // another device has a number of its own
  assert(kept(get) == 101 && kept(get) == 101 && asked == 2);
  current = 0;
  assert(kept(get) == 100 && asked == 2);
  current = 2;                                              // a failure is not kept
  assert(kept([](int) { return 0; }) == 0 && kept(get) == 102 && asked == 3);
  current = 1000;                                           // beyond the table: asked each time
  assert(kept(get) == 1100 && kept(get) == 1100 && asked == 5);
  moe::PerDevice shared;
  std::vector<std::thread> ts;
  for (int t = 0; t < 16; ++t)
    ts.emplace_back([&, t] {
      current = t % 4;
      for (int i = 0; i < 10000; ++i) assert(shared([](int dev) { return dev + 1; }) == t % 4 + 1);
    });
  for (auto& t : ts) t.join();
}
"""


def test_what_is_kept_per_device(tmp_path):
    """Settings of a kernel hold for one device: the host keeps them apart, also for threads that call together."""
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PER_DEVICE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    subprocess.run([shutil.which("g++"), "-std=c++17", "-O1", "-pthread", "-I" + _build.CSRC, "-I" + cuda, str(src), "-o", str(exe)],
                   check=True)
    subprocess.run([str(exe)], check=True)


def test_the_attention_opts_in_per_device():
    """No process-wide flag guards the shared-memory limit, which is set for one device at a time."""
    src = open(os.path.join(_build.CSRC, "moe_attn.cu")).read()
    assert "static bool" not in src and "static PerDevice" in src


@pytest.fixture
def toy(tmp_path, monkeypatch):
    """The build with its tools replaced by ones that make empty files."""
    tool = tmp_path / "tool"
    tool.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n')
    tool.chmod(0o755)
    out = tmp_path / "out"
    monkeypatch.setattr(_build, "BUILD", str(out))
    monkeypatch.setattr(_build, "LIB", str(out / "lib.so"))
    monkeypatch.setattr(_build, "BINDING", str(out / "binding.so"))
    monkeypatch.setattr(_build, "nvcc", lambda: str(tool))
    monkeypatch.setenv("CXX", str(tool))
    return out


def test_the_library_builds_without_torch(toy, monkeypatch):
    """The C library needs the CUDA toolkit alone; the binding is left out."""
    monkeypatch.setitem(__import__("sys").modules, "torch", None)          # importing it fails
    assert not _build.up_to_date()
    assert _build.build() == str(toy / "lib.so")
    assert (toy / "lib.so").exists() and not (toy / "binding.so").exists()
    assert _build.up_to_date()


def test_the_library_is_built_where_the_binding_fails(toy, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.raises(RuntimeError, match="binding"):
        _build.build()
    assert (toy / "lib.so").exists() and not _build.up_to_date()


def test_both_are_built_with_torch(toy):
    _build.build()
    assert (toy / "lib.so").exists() and (toy / "binding.so").exists() and _build.up_to_date()
