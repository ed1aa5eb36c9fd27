"""CPU test of the host state that launches from several threads share."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_skinny_gb300", "csrc")

PROGRAM = r"""
#include <thread>
#include <vector>
#include "q4k_device_once.h"
int main() {
  static q4k::DeviceOnce once;
  std::atomic<int> ran{0}, wrong{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&] {
      for (int i = 0; i < 2000; ++i)
        for (int dev : {0, 5, 63, 64, -1}) wrong += once.run(dev, 0, [&] { return ++ran, 0; }) != 0;
    });
  for (auto& t : threads) t.join();
  const int first = ran;   // in range: once a device and thread at most; out of range: every time
  if (wrong || first < 3 + 2 * 16000 || first > 3 * 8 + 2 * 16000) return 1;
  if (once.run(7, 0, [] { return 2; }) != 2 || once.run(7, 0, [] { return 0; }) != 0) return 2;   // a failure is not kept
  return once.run(7, 0, [] { return 3; });
}
"""


def test_once_a_device_under_the_thread_sanitizer(tmp_path):
    def build(text, name):
        src, exe = tmp_path / (name + ".cpp"), tmp_path / name
        src.write_text(text)
        r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=thread", "-I" + CSRC, str(src), "-o", str(exe)],
                           capture_output=True, text=True)
        return exe if r.returncode == 0 else None, r.stderr

    trivial, _ = build("#include <thread>\nint main() { std::thread([] {}).join(); }", "trivial")
    if trivial is None or subprocess.run([str(trivial)], capture_output=True).returncode != 0:
        pytest.skip("no thread sanitizer here")
    exe, log = build(PROGRAM, "once")
    assert exe is not None, log
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[:2000]


@pytest.mark.parametrize("source", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp"))))
def test_no_plain_flags_in_static_storage(source):
    """A flag that every calling thread reads and writes is atomic or held under a lock."""
    with open(os.path.join(CSRC, source), encoding="utf-8") as fh:
        code = re.sub(r"//[^\n]*", "", fh.read())
    for m in re.finditer(r"static bool \w+\[\d*\]", code):
        body = code[max(0, m.start() - 200):m.end() + 600]
        assert "lock_guard" in body, code[m.start():m.end() + 200]
