"""The check of the notes the attention kernel leaves for its join, compiled for
the host: a note that no CTA wrote (its wait gave up) never leads outside the
partial results."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "top_selection_dsa_gb300", "csrc")

SOURCE = r"""
#include <climits>
#include <cstdio>
#include "dsa_kv4_span.h"
int main() {
  const int ctas = 7;
  const int odd[] = {INT_MIN, INT_MIN + 1, -8, -1, 0, 1, 2, 3, 6, 7, 8, 1000, INT_MAX - 1, INT_MAX};
  for (int cta : odd)
    for (int n : odd)
      for (int which : odd) {
        const long long first = (long long)cta, last = (long long)cta + n - 1;
        const bool inside = first >= 0 && n >= 1 && last < ctas && which >= 0 && which < 2;
        if (dsa::span_noted(cta, n, which, ctas) != inside) {
          printf("%d %d %d\n", cta, n, which);
          return 1;
        }
      }
  return 0;
}
"""


def test_notes_outside_the_results_are_not_followed(tmp_path):
    src, exe = tmp_path / "span.cpp", tmp_path / "span"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_join_asks_before_it_reads():
    text = open(os.path.join(CSRC, "dsa_kv4_attn.cu")).read()
    join = text[text.index("kv4_join_kernel(const"):]
    read = join.index("p.spans[item]")
    asked = join.index("span_noted(")
    first_use = join.index("part_of = ")
    assert read < asked < first_use
