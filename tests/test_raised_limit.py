"""CPU test of the shared-memory limit that launches raise: threads that launch one kernel with different sizes, over a
fake of the attribute.  A launch fails if the attribute is below its size at that moment."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "raised_limit.h"

enum Error { kOk = 0, kInvalid = 1 };

static std::atomic<int> attribute;

static Error set(int v) {  // as the driver's call, some time passes on both sides of the change
    std::this_thread::sleep_for(std::chrono::microseconds(30));
    attribute = v;
    std::this_thread::sleep_for(std::chrono::microseconds(30));
    return kOk;
}

// What a cache of the limit without a lock does.
struct Separate {
    std::atomic<int> known{0};
    template <class Set>
    Error at_least(int, int v, Set s) {
        if (known.load() < v) {
            const Error e = s(v);
            if (e != kOk) return e;
            known.store(v);
        }
        return kOk;
    }
};

template <class Limit>
int failures() {
    int bad = 0;
    for (int round = 0; round < 60; ++round) {
        Limit limit;
        attribute = 0;
        std::atomic<int> failed{0}, go{0};
        std::vector<std::thread> threads;
        for (int t = 0; t < 6; ++t)
            threads.emplace_back([&, t] {
                ++go;
                while (go < 6) std::this_thread::yield();
                for (int k = 0; k < 4; ++k) {
                    const int size = 1000 + 100 * ((t * 5 + k * 3 + round) % 7);
                    if (limit.at_least(3, size, set) != kOk || attribute < size) ++failed;
                }
            });
        for (auto& t : threads) t.join();
        if (limit.at_least(3, 1600, set) != kOk || attribute < 1600) ++failed;  // and ever after
        bad += failed != 0;
    }
    return bad;
}

int main() {
    pkv::RaisedLimit limit;
    int calls = 0, last = 0;
    Error answer = kInvalid;
    auto count = [&](int v) { ++calls, last = v; return answer; };
    bool right = limit.at_least(0, 100, count) == kInvalid && calls == 1;   // an error comes back and is not remembered
    answer = kOk;
    right = right && limit.at_least(0, 100, count) == kOk && calls == 2 && last == 100;
    right = right && limit.at_least(0, 50, count) == kOk && limit.at_least(0, 100, count) == kOk && calls == 2;
    right = right && limit.at_least(0, 101, count) == kOk && calls == 3 && last == 101;
    right = right && limit.at_least(1, 60, count) == kOk && calls == 4 && last == 60;  // each device has its own
    right = right && limit.at_least(63, 1, count) == kOk && calls == 5;
    std::printf("%d %d %d\n", right ? 1 : 0, failures<pkv::RaisedLimit>(), failures<Separate>());
}
"""


def test_threads_with_different_sizes(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "limit.cpp"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "paged_kv_cache_slots_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O2", "-pthread", "-I", csrc, str(src), "-o", str(tmp_path / "limit")], check=True)
    out = subprocess.run([str(tmp_path / "limit")], check=True, capture_output=True, text=True, timeout=120).stdout.split()
    assert out[0] == "1"
    assert out[1] == "0", f"{out[1]} of 60 rounds failed"
    assert int(out[2]) > 0, "the fake does not show what separate steps do"
