"""How the attention-weights kernel's blocks share its work, and which parts its
second kernel adds: csrc/wq_weights_line.h itself, which both kernels run,
compiled for the host and held to what it has to do.  Every query tile that sees
a key of a pair is taken once, the parts of a pair that lies in several blocks
are all added, each once and in order, and no other is."""
import random
import subprocess

import pytest

from w8a8_int8_quantized_token_gb300 import build_lib

PAIR = 256

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "wq_weights_line.h"
using namespace wq;
int main() {
  WeightsLine a{};
  int blocks, cu;
  while (scanf("%d %d %d %d %d %d %d %d %d", &a.T, &a.B, &a.max_q, &a.heads, &a.max_len, &a.tpt, &a.shift, &blocks, &cu) == 9) {
    std::vector<int32_t> q(a.B + 1), l(a.B);
    if (cu) for (auto &v : q) if (scanf("%d", &v) != 1) return 1;
    for (auto &v : l) if (scanf("%d", &v) != 1) return 1;
    a.cu_q = cu ? q.data() : nullptr;
    a.key_len = l.data();
    auto cost = [&](int b) {
      const Seq s = seq_of(a, first_of(a, b), first_of(a, b + 1), a.key_len[b]);
      return s.before(s.pairs, a.shift) * a.heads;
    };
    int64_t total = 0;
    for (int b = 0; b < a.B; ++b) total += cost(b);
    auto place = [&](int64_t at) {
      Place p{0, at, total, at};
      while (at < total && p.off >= cost(p.b)) p.off -= cost(p.b), ++p.b;
      return p;
    };
    printf("problem %lld\n", (long long)total);
    for (int c = 0; c < blocks; ++c) {
      const Place at = place(first_unit(total, c, blocks));
      Walk w;
      w.begin(a, at, first_unit(total, c + 1, blocks) - at.at);
      for (Piece o; w.next(a, o);)
        printf("piece %d %d %d %d %d %d %d %d %d\n", c, o.b, o.h, o.k0, o.pairs, o.qa, o.qb, int(o.whole), o.slot);
    }
    for (int c = 0; c + 1 < blocks; ++c) {
      const Place at = place(first_unit(total, c + 1, blocks));
      Walk w;
      int64_t end;
      if (!left_to_others(a, at, c, blocks, w, end)) continue;
      printf("join %d %d %d %d", c, w.b, w.h, w.p);
      parts_after(total, c, blocks, end, [&](int64_t k) { printf(" %d", int(k)); });
      printf("\n");
    }
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("line")
    (at / "line.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", build_lib.CSRC,
                    str(at / "line.cpp"), "-o", str(at / "line")], check=True)
    return str(at / "line")


def problem(r):
    tpt, heads = r.choice([1, 2, 3, 16, 18, 25, 42, 64, 100, 128]), r.randint(1, 4)
    most = r.choice([1, 3, 40, 700, 3000])
    seqs = []
    for _ in range(r.randint(1, 9)):
        n = r.choice([0, 1, r.randint(1, most)])
        seqs.append((n, r.choice([0, n, max(0, n - r.randint(0, 9)), n + r.randint(0, 2000)])))
    if r.random() < 0.2:  # even tokens, no cu_q
        n = r.randint(1, most)
        seqs = [(n, k) for _, k in seqs]
    return tpt, heads, seqs, r.choice([1, 2, 3, 7, 40, 152])


def text(tpt, heads, seqs, blocks):
    n = [q for q, _ in seqs]
    even = len(set(n)) == 1 and n[0] > 0
    cu = [] if even else [sum(n[:b]) for b in range(len(n) + 1)]
    head = [sum(n), len(n), max(max(n), 1), heads, max(max(k for _, k in seqs), 1), tpt, tpt.bit_length() - 1, blocks, int(not even)]
    return " ".join(map(str, head + cu + [k for _, k in seqs]))


def hold(tpt, heads, seqs, blocks, lines):
    """lines: the program's words for this problem."""
    taken, parts, order = set(), {}, {}
    for w in lines:
        if w[0] != "piece":
            continue
        c, b, h, k0, pairs, qa, qb, whole, slot = map(int, w[1:])
        assert k0 % PAIR == 0 and (pairs == 1 or whole) and 0 <= qa <= qb
        for k in range(pairs):
            p = k0 // PAIR + k
            assert (k0 + k * PAIR) < seqs[b][1] and h < heads
            for q in range(qa, qb):
                assert (b, h, p, q) not in taken
                taken.add((b, h, p, q))
            if whole:
                assert ("whole", b, h, p) not in order
                order["whole", b, h, p] = c
            else:
                assert (c, slot) not in parts, "two parts in one place of the workspace"
                parts[c, slot] = (b, h, p)
                order.setdefault((b, h, p), []).append((c, slot))
    want, pairs = set(), set()
    for b, (n, length) in enumerate(seqs):
        tiles, old = -(-n // tpt), length - n
        for h in range(heads):
            for p in range(-(-length // PAIR)):
                pairs.add((b, h, p))
                # the last token of a tile sees key old + its place
                want |= {(b, h, p, q) for q in range(tiles) if tiles == 1 or old + min(n, (q + 1) * tpt) - 1 >= p * PAIR}
    assert taken == want
    # a pair's sums go to the weights by one block, or through the workspace: its first part to place 1, the others' to 0
    assert {k[1:] for k in order if k[0] == "whole"} | set(parts.values()) == pairs
    assert not {k[1:] for k in order if k[0] == "whole"} & set(parts.values())
    joined = {}
    for w in lines:
        if w[0] == "join":
            c, b, h, p, *others = map(int, w[1:])
            assert (b, h, p) not in joined
            joined[b, h, p] = [(c, 1)] + [(k, 0) for k in others]
    assert joined == {k: v for k, v in order.items() if k[0] != "whole"}
    return max((len(v) for v in joined.values()), default=0)


def split(out):
    found = []
    for line in out.splitlines():
        if line.startswith("problem"):
            found.append([])
        else:
            found[-1].append(line.split())
    return found


@pytest.mark.parametrize("seed", range(20))
def test_every_unit_is_taken_once_and_every_part_is_joined(program, seed):
    r = random.Random(seed)
    problems = [problem(r) for _ in range(40)]
    out = subprocess.run([program], input="\n".join(text(*p) for p in problems), capture_output=True, text=True, check=True)
    found = split(out.stdout)
    assert len(found) == len(problems)
    most = [hold(*p, lines) for p, lines in zip(problems, found)]
    assert max(most) > 3  # pairs that lie in more than three blocks are among them


# The cuts of some cases that run on a GPU (test_gpu_weights.py): tokens and keys, key heads, heads of one, blocks of a pair at most
@pytest.mark.parametrize("seqs,heads,G,most", [([(600, 700), (37, 900), (300, 300)], 2, 3, 4), ([(257, 1030)], 3, 6, 4), ([(70, 200), (129, 129)], 2, 2, 2)])
def test_cases_of_the_kernels_own_tests_cut_pairs(program, seqs, heads, G, most):
    max_q = max(n for n, _ in seqs)
    tpt = max(1, min(128 // G, max_q))
    units = len(seqs) * heads * -(-max(k for _, k in seqs) // PAIR) * max(1, -(-max_q // tpt))
    blocks = max(1, min(152, units))
    out = subprocess.run([program], input=text(tpt, heads, seqs, blocks), capture_output=True, text=True, check=True)
    assert hold(tpt, heads, seqs, blocks, split(out.stdout)[0]) >= most


def test_a_lengths_past_the_bounds_is_cut(program):
    """One token and one key too many by the host's bounds: both are cut."""
    out = subprocess.run([program], input="5 1 4 1 300 2 1 3 1 0 5 301", capture_output=True, text=True, check=True).stdout
    cut = subprocess.run([program], input="4 1 4 1 300 2 1 3 1 0 4 300", capture_output=True, text=True, check=True).stdout
    assert out == cut and "piece" in out
