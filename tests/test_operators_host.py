"""Refusals of the operators around the recurrent layers: every call here is
turned back by the checks of the C entry, before any CUDA work."""
import ctypes

import pytest
import torch

kda = pytest.importorskip("kda_gated_delta_chunked_gb300",
                          reason="libkda.so not built (run __graft_entry__.build())")

BAD, UNSUP, WS = kda.KDA_ERR_INVALID_ARGUMENT, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE


class Ptr:
    """Stands in for a tensor in a pointer slot; never dereferenced."""
    def __init__(self, addr):
        self.addr = addr

    def data_ptr(self):
        return self.addr

    def __add__(self, n):
        return Ptr(self.addr + n)


P = [Ptr((1 << 20) + i * (1 << 24)) for i in range(10)]


def test_struct_sizes_match_the_header(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    c = tmp_path / "s.c"
    c.write_text('#include <stdio.h>\n#include "kda.h"\nint main(void){printf("%zu %zu %zu %zu", sizeof(kda_norm_desc),'
                 'sizeof(kda_matmul_desc), sizeof(kda_latent_desc), offsetof(kda_latent_desc, workspace));return 0;}\n')
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(c), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    L = kda.KdaLatentDesc
    assert got == [ctypes.sizeof(kda.KdaNormDesc), ctypes.sizeof(kda.KdaMatmulDesc), ctypes.sizeof(L), L.workspace.offset]


def norm(d=None, x=P[0], w=P[1], r=P[2], h=P[3], y=P[4], q=P[5], s=P[6], **kw):
    f = dict(rows=10, dim=256, dtype=kda.KDA_BF16, x_stride=256, residual_stride=256, eps=1e-6)
    f.update(kw)
    return kda.kda_rms_norm(kda.KdaNormDesc(**f), x, w, r, h, y, q, s, 0)


def test_norm_refusals():
    assert norm(rows=-1) == BAD and norm(dim=0) == BAD and norm(dtype=2) == BAD
    assert norm(x_stride=255) == BAD and norm(residual_stride=255) == BAD
    assert norm(eps=-1.0) == BAD and norm(eps=float("nan")) == BAD and norm(eps=float("inf")) == BAD
    assert norm(q=None) == BAD and norm(s=None) == BAD                       # both or neither
    assert norm(x=None) == BAD and norm(h=None, y=None, q=None, s=None) == BAD
    assert norm(x=P[0] + 1) == BAD and norm(s=P[6] + 2) == BAD
    assert norm(y=P[0] + 512) == BAD and norm(q=P[2]) == BAD and norm(y=P[3]) == BAD and norm(y=P[1]) == BAD
    assert norm(h=P[0] + 512) == BAD and norm(h=P[0], x_stride=300) == BAD    # in place only exactly
    assert norm(rows=1 << 31, dim=1, x_stride=1, residual_stride=1) == UNSUP
    assert norm(rows=0, x=None, h=None, y=None, q=None, s=None) == kda.KDA_OK


def matmul(a=P[0], sa=P[1], b=P[2], sb=P[3], c=P[4], **kw):
    f = dict(m=10, n=300, k=256, a_stride=256, b_stride=256, c_stride=300, dtype=kda.KDA_BF16, flags=0)
    f.update(kw)
    return kda.kda_matmul_fp8(kda.KdaMatmulDesc(**f), a, sa, b, sb, c, 0)


def test_matmul_refusals():
    assert matmul(m=-1) == BAD and matmul(n=-1) == BAD and matmul(k=0) == BAD and matmul(dtype=7) == BAD
    assert matmul(a_stride=255) == BAD and matmul(b_stride=255) == BAD and matmul(c_stride=299) == BAD
    assert matmul(flags=2) == BAD
    assert matmul(a=None) == BAD and matmul(sa=None) == BAD and matmul(b=None) == BAD and matmul(sb=None) == BAD
    assert matmul(c=None) == BAD and matmul(c=P[4] + 1) == BAD and matmul(sa=P[1] + 2) == BAD
    assert matmul(c=P[0] + 64) == BAD and matmul(c=P[1]) == BAD
    assert matmul(m=1 << 31) == UNSUP
    assert matmul(m=0, a=None, c=None) == kda.KDA_OK and matmul(n=0, c_stride=0, b=None) == kda.KDA_OK


def latent(**kw):
    f = dict(num_seqs=2, num_heads=4, dtype=kda.KDA_BF16, flags=0, scale=0.1, d_k=128, d_rope=64, d_v=128, total_q=50, total_k=60,
             q_token_stride=768, q_head_stride=192, k_token_stride=512, k_head_stride=128, v_token_stride=512, v_head_stride=128,
             rope_token_stride=64, workspace=P[9].addr, workspace_bytes=1 << 24)
    f.update(kw)
    return kda.KdaLatentDesc(**f)


def prefill(q=P[0], k=P[1], r=P[2], v=P[3], cq=P[4], ck=P[5], out=P[6], lse=P[7], **kw):
    return kda.kda_latent_prefill(latent(**kw), q, k, r, v, cq, ck, out, lse, 0)


def test_prefill_refusals():
    assert prefill(num_seqs=-1) == BAD and prefill(num_heads=0) == BAD and prefill(dtype=3) == BAD and prefill(flags=8) == BAD
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert prefill(scale=s) == BAD
    assert prefill(d_k=0) == BAD and prefill(d_rope=-1) == BAD and prefill(d_v=0) == BAD and prefill(total_q=-1) == BAD
    assert prefill(d_k=200) == UNSUP and prefill(d_v=257) == UNSUP and prefill(num_heads=70000) == UNSUP
    assert prefill(q_token_stride=-1) == BAD
    assert prefill(cq=None) == BAD and prefill(cq=None, ck=None) == BAD          # no lengths: one sequence only
    assert prefill(q=None) == BAD and prefill(k=None) == BAD and prefill(r=None) == BAD and prefill(out=None) == BAD
    assert prefill(d_rope=0) == BAD                                               # a rotary key without channels
    assert prefill(q=P[0] + 1) == BAD and prefill(lse=P[7] + 2) == BAD and prefill(cq=P[4] + 1) == BAD
    assert prefill(out=P[3]) == BAD and prefill(lse=P[6]) == BAD and prefill(out=P[9]) == BAD
    assert prefill(workspace=None) == WS and prefill(workspace_bytes=8) == WS and prefill(workspace=P[9].addr + 8) == WS
    assert prefill(num_seqs=0) == kda.KDA_OK and prefill(total_q=0, q=None, out=None) == kda.KDA_OK


def decode(q=P[0], cache=P[1], table=P[2], lens=P[3], out=P[4], lse=P[5], **kw):
    f = dict(d_k=512, d_rope=64, d_v=512, q_token_stride=4 * 576, q_head_stride=576, num_queries=1, page_size=64, num_pages=10,
             max_pages=5, page_stride=64 * 576)
    f.update(kw)
    return kda.kda_latent_decode(latent(**f), q, cache, table, lens, out, lse, 0)


def test_decode_refusals():
    assert decode(num_queries=0) == BAD and decode(page_size=0) == BAD and decode(max_pages=0) == BAD and decode(num_pages=-1) == BAD
    assert decode(d_v=256) == BAD and decode(page_stride=64 * 576 - 1) == BAD and decode(flags=kda.KDA_FLAG_NO_CAUSAL) == BAD
    assert decode(d_k=513, d_v=513, page_stride=64 * 577) == UNSUP and decode(d_rope=129, page_stride=64 * 641) == UNSUP
    assert decode(max_pages=1 << 30) == UNSUP
    assert decode(q=None) == BAD and decode(cache=None) == BAD and decode(table=None) == BAD and decode(lens=None) == BAD
    assert decode(out=None) == BAD and decode(out=P[4] + 1) == BAD and decode(table=P[2] + 2) == BAD
    assert decode(out=P[1] + 64) == BAD and decode(lse=P[0]) == BAD and decode(out=P[9] + 64) == BAD
    assert decode(workspace=None) == WS and decode(workspace_bytes=8) == WS
    assert decode(num_seqs=0) == kda.KDA_OK
    d = latent(d_k=512, d_v=512, num_queries=1, page_size=64, num_pages=10, max_pages=5, page_stride=64 * 576)
    assert kda.kda_latent_decode_workspace_bytes(d) > 0 and kda.kda_latent_prefill_workspace_bytes(d) == 0


def test_python_refusals():
    """What the torch layer turns back: here, anything that is not on a CUDA device."""
    x = torch.zeros(4, 256)
    for call in (lambda: kda.rms_norm(x), lambda: kda.matmul_fp8(x, x, x, x), lambda: kda.latent_prefill(x, x, x, x, scale=1.0),
                 lambda: kda.latent_decode(x, x, x, x, scale=1.0)):
        with pytest.raises(ValueError):
            call()


PER_DEVICE = r'''
#include <cstdio>
#include <thread>
#include <vector>
#include "kda_per_device.h"

enum Error { kGood = 0, kBad = 2 };

int main() {
    static kda::PerDevice one;
    int out = 0;
    std::atomic<int> asked{0};
    auto is = [&](int n) { return [&asked, n](int& x) { ++asked; x = n; return kGood; }; };
    if (one.get(0, out, [](int& x) { x = 9; return kBad; }) != kBad) return 1;           // an error is not kept
    if (one.get(0, out, is(5)) != kGood || out != 5 || asked != 1) return 2;
    if (one.get(0, out, is(6)) != kGood || out != 5 || asked != 1) return 3;             // found before
    if (one.get(1, out, is(7)) != kGood || out != 7 || asked != 2) return 4;             // another device
    if (one.get(0, out, is(8)) != kGood || out != 5) return 5;
    if (one.get(100, out, is(3)) != kGood || out != 3 || one.get(100, out, is(4)) != kGood || out != 4) return 6;   // beyond those kept
    static kda::PerDevice two;
    std::vector<std::thread> all;
    std::atomic<int> wrong{0};
    for (int t = 0; t < 16; ++t)
        all.emplace_back([&, t] {
            for (int i = 0; i < 2000; ++i) {
                int x = 0;
                if (two.get(i % 64, x, [i](int& n) { n = 1 + i % 64; return kGood; }) != kGood || x != 1 + i % 64) ++wrong;
            }
        });
    for (auto& t : all) t.join();
    return wrong ? 7 : 0;
}
'''


def test_what_is_found_for_a_device_is_kept_for_it_alone(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "d.cpp").write_text(PER_DEVICE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", os.path.join(root, "kda_gated_delta_chunked_gb300", "csrc"),
                    str(tmp_path / "d.cpp"), "-o", str(tmp_path / "d")], check=True)
    assert subprocess.run([str(tmp_path / "d")]).returncode == 0


def test_nothing_of_a_device_is_kept_for_the_process():
    """Functions' plain statics would be the first device's: attributes of kernels, blocks that run at once."""
    import glob
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for name in ("kda_norm.cu", "kda_matmul_tc.cu", "kda_latent_prefill_tc.cu", "kda_latent_decode_tc.cu"):
        path, = glob.glob(os.path.join(root, "kda_gated_delta_chunked_gb300", "csrc", name))
        found = re.findall(r"^ {4,}static (?!constexpr|__device__)(\w+)", open(path).read(), re.M)
        assert set(found) <= {"PerDevice", "uint32_t"}, (name, found)     # (uint32_t: a member function)


IMPORT = '''
import sys
sys.path.insert(0, sys.argv[1])
import torch
import kda_gated_delta_chunked_gb300 as kda
assert kda.kda_status_string(kda.KDA_OK) == "KDA_OK" and kda.prefill and kda.decode_step
d = kda.make_desc(1, 1, 128, 128, 64, torch.bfloat16, None)
assert kda.kda_prefill_workspace_bytes(d) > 0
x = torch.zeros(4, 256)
for call in (lambda: kda.rms_norm(x), lambda: kda.matmul_fp8(x, x, x, x)):
    try:
        call()
    except (ImportError, ValueError) as e:
        print(type(e).__name__)
'''


def test_the_other_calls_do_without_the_module_for_torch_tensors(tmp_path):
    """Without it, or with one that this Python cannot load, the package imports, its other calls work, and the operators
    say what is missing.  KDA_LIBRARY leads to the module beside that library, if there is one."""
    import os
    import shutil
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    package, built = "kda_gated_delta_chunked_gb300", kda.library_path()
    other = tmp_path / "other"
    (tmp_path / package / "_build").mkdir(parents=True)
    other.mkdir()
    for f in os.listdir(os.path.join(root, package)):
        if f.endswith(".py"):
            shutil.copy(os.path.join(root, package, f), tmp_path / package / f)
    for to in (tmp_path / package / "_build", other):
        shutil.copy(built, to / "libkda.so")

    def names(**env):
        r = subprocess.run([sys.executable, "-c", IMPORT, str(tmp_path)], capture_output=True, text=True, timeout=300,
                           env={**{k: v for k, v in os.environ.items() if k != "KDA_LIBRARY"}, **env})
        assert r.returncode == 0, r.stderr[-1500:]
        return r.stdout.split()
    module = os.path.join(root, package, "_build", "_kda_torch.so")
    assert names() == ["ImportError"] * 2
    (tmp_path / package / "_build" / "_kda_torch.so").write_bytes(b"not a module")
    assert names() == ["ImportError"] * 2
    shutil.copy(module, other / "_kda_torch.so")
    assert names(KDA_LIBRARY=str(other / "libkda.so")) == ["ValueError"] * 2          # loaded: the tensors are not on a GPU
    shutil.copy(module, tmp_path / package / "_build" / "_kda_torch.so")
    (other / "_kda_torch.so").unlink()
    assert names(KDA_LIBRARY=str(other / "libkda.so")) == ["ValueError"] * 2 and names() == ["ValueError"] * 2


def test_the_module_for_torch_tensors_is_built_anew_for_another_python_or_torch(tmp_path, monkeypatch):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(kda.__file__), "build.py")
    spec = importlib.util.spec_from_file_location("_kda_build_test", path)
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    src = os.path.join(build.CSRC, "kda_torch.cpp")
    assert not build._torch_module_stale(src)                       # as the package was built
    with open(build.TORCH_MODULE + ".for") as f:
        mark = f.read()
    monkeypatch.setattr(build, "TORCH_MODULE", str(tmp_path / "m.so"))
    assert build._torch_module_stale(src)                           # none
    (tmp_path / "m.so").write_bytes(b"")
    assert build._torch_module_stale(src)                           # one that does not say what it is for
    (tmp_path / "m.so.for").write_text(mark)
    assert not build._torch_module_stale(src)
    for other in (mark.replace(torch.__version__, "2.0.0"), "another Python\n" + mark):
        assert other != mark
        (tmp_path / "m.so.for").write_text(other)
        assert build._torch_module_stale(src)
