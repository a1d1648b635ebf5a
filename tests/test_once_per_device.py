"""csrc/once.h on the host, with a stand-in for the CUDA runtime's two names
that it uses: threads whose first calls meet, a setup that fails, devices kept
apart."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUNTIME = """
#pragma once
enum cudaError_t { cudaSuccess = 0, cudaErrorInvalidDevice = 101, cudaErrorUnknown = 999 };
extern thread_local int g_device;
inline cudaError_t cudaGetDevice(int *d) { *d = g_device; return cudaSuccess; }
"""

MAIN = r"""
#include "once.h"
#include <cstdio>
#include <thread>
#include <vector>

thread_local int g_device = 0;
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)

int main() {
    for (int round = 0; round < 200; ++round) {  // no thread gets past it with a value unset
        moe::OncePerDevice once;
        std::atomic<int> units[2] = {}, wrong{0}, go{0};
        std::vector<std::thread> ts;
        for (int t = 0; t < 8; ++t)
            ts.emplace_back([&] {
                ++go;
                while (go < 8) {}
                const cudaError_t e = once([&](int) {
                    units[0].store(152, std::memory_order_relaxed);
                    units[1].store(76, std::memory_order_relaxed);
                    return cudaSuccess;
                });
                if (e != cudaSuccess || units[0].load(std::memory_order_relaxed) != 152 ||
                    units[1].load(std::memory_order_relaxed) != 76)
                    ++wrong;
            });
        for (auto &t : ts) t.join();
        CHECK(wrong == 0);
    }
    moe::OncePerDevice once;
    int calls = 0;
    auto setup = [&](int d) { ++calls; return calls == 1 ? cudaErrorUnknown : d == g_device ? cudaSuccess : cudaErrorInvalidDevice; };
    CHECK(once(setup) == cudaErrorUnknown);  // and is tried again
    CHECK(once(setup) == cudaSuccess && calls == 2);
    CHECK(once(setup) == cudaSuccess && calls == 2);
    g_device = 5;
    CHECK(once(setup) == cudaSuccess && calls == 3);
    CHECK(once(setup) == cudaSuccess && calls == 3);
    for (int d : {-1, 64}) {
        g_device = d;
        CHECK(once(setup) == cudaErrorInvalidDevice && calls == 3);
    }
    return 0;
}
"""


def test_once_per_device(tmp_path):
    (tmp_path / "cuda_runtime.h").write_text(RUNTIME)
    (tmp_path / "main.cc").write_text(MAIN)
    exe = tmp_path / "once"
    csrc = os.path.join(ROOT, "token_dispatch_grouped_fp32_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-pthread", f"-I{tmp_path}", f"-I{csrc}",
                    str(tmp_path / "main.cc"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
