"""What is asked of a device once (csrc/per_device.cuh), compiled with the host
compiler and driven with made-up queries, on the CPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.cuh"

enum Error { kNone = 0, kFailed = 7 };
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

struct Limits { int sms, clusters; };

int main() {
    static ep::PerDevice<Limits, 8> table;
    int asked = 0;
    auto query = [&](int device, Error result) {
        return [&asked, device, result](Limits* v) {
            ++asked;
            *v = {100 + device, 10 * device};  // (also where it fails)
            return result;
        };
    };
    Limits v{};
    // a failure is passed on, leaves the caller's value alone and is not kept
    v = {-1, -1};
    CHECK(table.get(3, &v, query(9, kFailed)) == kFailed && asked == 1);
    CHECK(v.sms == -1);
    CHECK(table.get(3, &v, query(3, kNone)) == kNone && asked == 2 && v.sms == 103);
    // asked once for each device
    for (int i = 0; i < 3; ++i)
        for (int d = 0; d < 8; ++d) {
            v = {-1, -1};
            CHECK(table.get(d, &v, query(d, kNone)) == kNone);
            CHECK(v.sms == 100 + d && v.clusters == 10 * d);
        }
    CHECK(asked == 2 + 7);
    // kept: a later query is not made, whatever it would say
    CHECK(table.get(5, &v, query(6, kFailed)) == kNone && v.sms == 105 && asked == 9);
    // ordinals outside the table are asked each time
    for (int d : {-1, 8, 1000}) {
        CHECK(table.get(d, &v, query(d, kNone)) == kNone && v.sms == 100 + d);
        CHECK(table.get(d, &v, query(d, kFailed)) == kFailed);
    }
    CHECK(asked == 15);
    // many threads, every device: one query each, every reader sees its result
    static ep::PerDevice<Limits, 8> shared;
    std::atomic<int> queries{0}, wrong{0};
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&, t] {
            for (int i = 0; i < 2000; ++i) {
                const int d = (t + i) % 8;
                Limits got{};
                const Error e = shared.get(d, &got, [&](Limits* out) {
                    ++queries;
                    *out = {d, d + 1};
                    return kNone;
                });
                if (e != kNone || got.sms != d || got.clusters != d + 1) ++wrong;
            }
        });
    for (auto& t : threads) t.join();
    CHECK(queries == 8 && wrong == 0);
    std::puts("ok");
    return 0;
}
"""


def test_values_per_device(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "combine_movement_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", inc, str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_products_keep_nothing_for_the_process():
    """Which split of K a product takes goes by its device; a table that is
    filled once for the process would give a second device the first one's."""
    with open(os.path.join(ROOT, "combine_movement_gb300", "csrc", "expert_fp8.cu")) as f:
        text = f.read()
    statics = [line.strip() for line in text.splitlines() if line.strip().startswith("static ")
               and not line.strip().startswith("static_assert")]
    assert statics and all("PerDevice<" in s or "EncodeFn> known" in s for s in statics), statics
