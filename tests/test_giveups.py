"""The host's account of device waits that gave up (csrc/giveups.h), compiled here with g++: each is
reported once, whatever is written while a caller reads."""
import shutil
import subprocess

import pytest

from prefill_only_decision_gb300 import build

SRC = r"""
#include "giveups.h"
#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
  {
    s1::GiveUps<2> g;
    uint64_t word[2] = {0, 0};
    bool any = false;
    auto read = [&](uint64_t* now) { now[0] = word[0]; now[1] = word[1]; return 0; };
    auto news = [&](int dev) { CHECK(g.news(dev, read, &any) == 0); return any ? 2 : 0; };
    CHECK(news(0) == 0);
    word[0] = 1000;
    CHECK(news(0) == 2 && news(0) == 0 && news(1) == 2 && news(1) == 0);   // once for each device
    word[1] = 900;                                                         // the other kernel's word alone
    CHECK(news(0) == 2 && news(0) == 0);
    word[0] = 999;                                                         // written after a later time
    CHECK(news(0) == 2 && news(0) == 0);
    // written while a caller reads: not in what it has read, so the next call's
    auto late = [&](uint64_t* now) { read(now); word[1] = 2000; return 0; };
    CHECK(g.news(0, late, &any) == 0 && !any && news(0) == 2 && news(0) == 0);
    // a reading that fails tells nothing
    word[0] = 3000;
    CHECK(g.news(0, [](uint64_t*) { return 7; }, &any) == 7 && news(0) == 2 && news(0) == 0);
  }
  {   // four callers while a device writes
    s1::GiveUps<1> g;
    std::atomic<uint64_t> word{0};
    std::atomic<int> told{0};
    const int N = 20000;
    auto read = [&](uint64_t* now) { *now = word.load(); return 0; };
    std::vector<std::thread> t;
    for (int i = 0; i < 4; ++i)
      t.emplace_back([&] {
        for (bool last = false; !last;) {
          last = word.load() == (uint64_t)N;
          bool any = false;
          g.news(0, read, &any);
          if (any) ++told;
        }
      });
    for (int i = 0; i < N; ++i) ++word;
    for (auto& x : t) x.join();
    bool any = true;
    CHECK(told >= 1 && told <= N && g.news(0, read, &any) == 0 && !any);
  }
  return 0;
}
"""


def test_give_ups(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(SRC)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I" + build.CSRC, str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
