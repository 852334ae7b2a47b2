"""Host state that all callers share: calls from several threads at once."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemv_quantize_q8_gb300", "csrc")

LOOKUPS = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "kq_lookup.cuh"
int main() {
    static std::atomic<int> slots[64];
    std::atomic<int> wrong{0};
    std::vector<std::thread> all;
    for (int t = 0; t < 8; ++t)
        all.emplace_back([&] {
            for (int i = 0; i < 64; ++i)
                if (kq::looked_up(slots[i], [i] { return 100 + i; }) != 100 + i) ++wrong;
        });
    for (auto &t : all) t.join();
    return wrong.load() ? 1 : 0;
}
"""


def test_lookups_are_no_data_race(tmp_path):
    """The per-device lookups' slots under the thread sanitizer, asked by eight threads at once."""
    src, exe = tmp_path / "lookups.cc", tmp_path / "lookups"
    src.write_text(LOOKUPS)
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fsanitize=thread", "-I", CSRC, str(src), "-o", str(exe), "-lpthread"]
    built = subprocess.run(cmd, capture_output=True, text=True)
    if built.returncode and "tsan" in built.stderr:
        pytest.skip("no thread sanitizer here")
    assert built.returncode == 0, built.stderr
    ran = subprocess.run([str(exe)], capture_output=True, text=True)
    if "unexpected memory mapping" in ran.stderr:
        pytest.skip("the thread sanitizer does not run under this kernel")
    assert ran.returncode == 0 and "data race" not in ran.stderr, ran.stderr


def test_every_shared_lookup_is_atomic():
    """No function keeps a plain variable from call to call where a lookup is cached."""
    for name in sorted(os.listdir(CSRC)):
        for line in open(os.path.join(CSRC, name)):
            text = line.split("//")[0]
            assert not ("cache[" in text and "static" in text and "std::atomic" not in text), f"{name}: {line.strip()}"


THREADS = r"""
import threading
import torch
import gemv_quantize_q8_gb300 as kq
sizes = [(M, N, K) for M in (12, 50, 100, 300) for N, K in ((300, 2048), (1000, 640))]
torch.cuda.init()
made = []
for i, (M, N, K) in enumerate(sizes):
    g = torch.Generator(device="cuda")
    g.manual_seed(i)
    q, w = (torch.randint(-128, 128, (r, K), generator=g, device="cuda", dtype=torch.int8) for r in (M, N))
    n = kq.kq_gemm_i8_workspace_bytes(M, N, K)
    made.append((q, w, torch.ones(M, device="cuda"), torch.ones(N, device="cuda"), torch.zeros((M, N), device="cuda"),
                 torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
torch.cuda.synchronize()
gate = threading.Barrier(len(sizes))
def work(i):
    (M, N, K), (q, w, sx, sw, y, ws, stream) = sizes[i], made[i]
    gate.wait()
    for _ in range(5):
        kq.kq_gemm_i8(q, K, sx, w, K, sw, None, M, N, K, kq.F32, y, N, ws, ws.numel(), stream=stream)
threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
for (M, N, K), (q, w, sx, sw, y, ws, stream) in zip(sizes, made):
    assert torch.equal(y.double(), q.double() @ w.double().T), (M, N, K)
    assert kq.kq_read_device_flag(ws) == 0
print("all right")
"""


@pytest.mark.gpu
def test_first_calls_of_several_threads():
    """The first tensor-core products of a process, of every form, from eight threads on streams of their own."""
    ran = subprocess.run([sys.executable, "-c", THREADS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert ran.returncode == 0 and "all right" in ran.stdout, ran.stderr[-2000:]
