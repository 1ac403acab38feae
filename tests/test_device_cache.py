"""What the host remembers of a device (csrc/device_cache.h), on the CPU: each
device has its own answers, and a question that failed is asked again."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_routing_mxfp4_gb300", "csrc")

MAIN = r"""
#include <cassert>
#include <thread>
#include <vector>
#include "device_cache.h"
int main()
{
    static lmoe::DeviceCache<4> c;
    int asked = 0;
    auto answer = [&](int v) { return [&asked, v] { ++asked; return v; }; };
    assert(c.get(0, 2, answer(0)) == 0 && c.get(0, 2, answer(-5)) == 0);  // failed, twice
    assert(c.get(0, 2, answer(37)) == 37 && asked == 3);
    assert(c.get(0, 2, answer(99)) == 37 && asked == 3);      // remembered
    assert(c.get(1, 2, answer(18)) == 18 && asked == 4);      // another device
    assert(c.get(0, 3, answer(9)) == 9 && asked == 5);        // another question
    for (int dev : {-1, c.DEVICES, 1 << 20}) {                // a device it has no room for: asked each time
        assert(c.get(dev, 2, answer(7)) == 7 && c.get(dev, 2, answer(8)) == 8);
    }
    assert(asked == 11 && c.get(0, 2, answer(1)) == 37);
    std::vector<std::thread> t;
    for (int i = 0; i < 8; ++i) t.emplace_back([] { for (int k = 0; k < 1000; ++k) assert(c.get(3, 1, [] { return 5; }) == 5); });
    for (auto &x : t) x.join();
}
"""


def test_device_cache(tmp_path):
    src = tmp_path / "main.cpp"
    src.write_text(MAIN)
    exe = tmp_path / "main"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", f"-I{CSRC}", str(src), "-o", str(exe)],
                   check=True)
    subprocess.run([str(exe)], check=True)


def test_the_linears_clusters_are_asked_for_through_it():
    src = open(os.path.join(CSRC, "k_linear_mxfp4.cu")).read()
    assert "DeviceCache<MAX_KS + 1>" in src and "static std::atomic<int> known" not in src
