"""Index arithmetic of the kernels (csrc/ds_index.h) on the CPU: every address that it gives lies in what the call was
given. The program is built so that a signed overflow ends it."""
import subprocess

import pytest

from vocab_wide_logit_gb300 import build


@pytest.fixture
def run(tmp_path):
    """Builds and runs a C++ program around the header; it returns 0 or prints what it found."""
    def go(body):
        src, exe = tmp_path / "t.cpp", str(tmp_path / "t")
        src.write_text('#include <cstdio>\n#include <algorithm>\n#include "ds_index.h"\nusing namespace ds;\n' + body)
        subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow",
                        "-fsanitize-undefined-trap-on-error", "-I", build.CSRC, str(src), "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout[-2000:] or r.returncode
    return go


def test_adapter_weights_by_words(run):
    """k_adapters_down reads an adapter's weights by words where rows start anywhere: blocks of 32 ranks up to R filled up
    to 16, 32, 64 or 128, eight inputs a lane and step. Every word holds an input that counts, every input is in one."""
    run(r"""
int main() {
  int bad = 0;
  for (int R = 1; R <= 128; ++R)
    for (int K : {1, 5, 7, 8, 33, 40, 97})
      for (int front = 0; front < 8; ++front)  // elements between a 16-byte boundary and the stack
        for (int a = 0; a < 3; ++a) {
          const int padded = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128;
          for (int rank = 0; rank < std::max(padded, 32); ++rank) {
            const int end = rank < R ? K : 0;
            for (int i = 0; i < (K + 31) / 32 * 32; i += 8) {
              const long long at = front + rank_at(a, rank, R, K) + i, word = at >> 1;
              const int odd = (int)(at & 1);
              unsigned seen = 0;
              for (int j = 0; j < 5; ++j) {
                if (!word_wanted(i, j, odd, end)) continue;
                int counts = 0;
                for (int e = 0; e < 2; ++e) {
                  const long long k = 2 * (word + j) + e - at;  // of the eight
                  if (k >= 0 && k < 8 && i + k < end) ++counts, seen |= 1u << k;
                }
                if (!counts && bad++ < 5) printf("R %d K %d front %d a %d rank %d i %d: word %d\n", R, K, front, a, rank, i, j);
              }
              const int some = std::max(0, std::min(8, end - i));
              if (seen != (1u << some) - 1 && bad++ < 5) printf("R %d K %d rank %d i %d: %x of %d\n", R, K, rank, i, seen, some);
            }
          }
        }
  return bad != 0;
}
""")


def test_ranks_that_fill_up_stay_in_the_stack(run):
    """Where a rank's inputs start is within the stack for every rank that a launch has, and exact beyond 32 bits."""
    run(r"""
int main() {
  int bad = 0;
  for (int R = 1; R <= 128; ++R)
    for (int K : {1, 1001, 1 << 30})
      for (int L : {1, 2, 8192}) {
        const int padded = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128;
        for (int rank = 0; rank < std::max(padded, 32); ++rank) {
          const long long at = rank_at(L - 1, rank, R, K), first = (long long)(L - 1) * R * K;
          if ((at < first || at >= first + (long long)R * K || (rank < R && at != first + (long long)rank * K)) && bad++ < 5)
            printf("R %d K %d L %d rank %d: %lld\n", R, K, L, rank, at);
        }
      }
  return bad != 0;
}
""")


def test_logits_in_front_of_a_token(run):
    """The ties in front of a token in its own chunk, a lane each: the right ones and none beside the row, for the last tokens
    of rows of every length up to the largest and every place of a row in its first chunk, and without a token."""
    run(r"""
int main() {
  int bad = 0;
  for (int E : {4, 8})
    for (int dc = 0; dc < E; ++dc)
      for (long long V : {1LL, 2LL, 40LL, 1025LL, 1LL << 30, (1LL << 31) - 64, (1LL << 31) - 33, (1LL << 31) - 9, (1LL << 31) - 8, (1LL << 31) - 2,
                          (1LL << 31) - 1})
        for (long long t = std::max(-1LL, V - 70); t < V; ++t) {
          const int token = (int)t, chunk = token < 0 ? 0 : chunk_of(token, E, dc);
          const int first = first_in_chunk(chunk, E, dc);
          const long long start = std::max(0LL, (long long)chunk * E - dc);
          bool wrong = first != start || (token >= 0 && (token < start || token >= (long long)(chunk + 1LL) * E - dc));
          for (int lane = 0; lane < 32; ++lane) {
            const bool in = in_front_of(token, first, lane);
            wrong |= in != (start + lane < token) || (in && start + lane >= V);
          }
          if (wrong && bad++ < 5) printf("E %d dc %d V %lld token %lld\n", E, dc, V, t);
        }
  return bad != 0;
}
""")


def test_logits_of_a_rows_chunks(run):
    """Which chunks a row has, what of a chunk is the row's, and where in it the token is: the first and last chunks of rows of
    every length up to the largest, at every place of a row in its first chunk; one chunk behind the row as a launch may have."""
    run(r"""
int main() {
  int bad = 0;
  for (int E : {4, 8})
    for (int dc = 0; dc < E; ++dc)
      for (long long back = 0; back < 64; ++back)
        for (long long V : {1 + back, (1LL << 30) - back, (1LL << 31) - 1 - back}) {
          const long long chunks = (V + 2 * E - 2) / E;  // of a launch
          for (long long q = 0; q < chunks; q = q == 4 && chunks > 9 ? chunks - 5 : q + 1) {
            const long long id = q * E - dc;
            bool wrong = (q < chunks_of((int)V, E, dc)) != (id < V);
            if (id < V) {
              const int first = first_of_chunk((unsigned)q, E, dc);
              int all = 0;
              for (int i = 0; i < E; ++i) {
                const bool in = id + i >= 0 && id + i < V;
                all += in;
                wrong |= in_row(first, i, (int)V) != in;
              }
              wrong |= first != id || all_in_row(first, E, (int)V) != (all == E);
              for (long long t : {0LL, 1LL, V / 2, V - 9, V - 8, V - 2, V - 1})
                if (t >= 0) {
                  const unsigned place = place_of((int)t, first);
                  wrong |= t >= id && t < id + E ? place != t - id : place < (unsigned)E;
                }
            }
            if (wrong && bad++ < 5) printf("E %d dc %d V %lld chunk %lld\n", E, dc, V, q);
          }
        }
  return bad != 0;
}
""")
