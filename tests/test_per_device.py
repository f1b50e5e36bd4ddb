"""csrc/per_device.h on the host, and who uses it: limits set with cudaFuncSetAttribute hold for one device."""
import os
import re
import subprocess

from tests.test_kv4_source import CSRC, source

PROGRAM = r"""
#include "per_device.h"
#include <thread>
#include <vector>
int main()
{
    static nm::OncePerDevice once;
    int calls[3] = {};
    bool works = true;
    const auto on = [&](int d) { return once(d, [&] { ++calls[d]; return works; }); };
    if (!on(0) || !on(0) || calls[0] != 1) return 1;          // once on a device
    if (!on(1) || calls[1] != 1 || !on(0) || calls[0] != 1) return 2; // and once on the next
    works = false;
    if (on(2) || on(2) || calls[2] != 2) return 3;            // a failure is tried again
    works = true;
    if (!on(2) || !on(2) || calls[2] != 3) return 4;
    if (once(-1, [] { return true; }) || once(nm::kMaxDevices, [] { return true; })) return 5;
    std::atomic<int> n{0};
    static nm::OncePerDevice many;
    std::vector<std::thread> t;
    for (int i = 0; i < 8; ++i) t.emplace_back([&] { for (int k = 0; k < 1000; ++k) if (!many(7, [&] { ++n; return true; })) n = -100; });
    for (auto &x : t) x.join();
    return n >= 1 && n <= 8 ? 0 : 6;
}
"""


def test_once_per_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_cache_keeps_no_device_state_for_the_process():
    for name in sorted(os.listdir(CSRC)):
        if not name.startswith("kv4"):
            continue
        text = source(name)
        assert "once_flag" not in text and "call_once" not in text, name
        for kind in re.findall(r"\n    +static (?!constexpr|_assert)(?!const )([\w:<>]+)", text):
            assert kind in ("OncePerDevice", "std::atomic<int>"), (name, kind)
        for at in re.finditer("cudaFuncSetAttribute", text):
            assert "OncePerDevice" in text[max(0, at.start() - 300):at.start()], name
