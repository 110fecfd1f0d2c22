// ds_index.h -- index arithmetic of kernels that the CPU tests go through at the sizes where it can go wrong. Plain C++:
// a host compiler takes it too.
#pragma once

namespace ds {

// ---------------------------------------------------------------- weights of an adapter, by words
// Where the K inputs of rank number `rank` of adapter a start in a stack [L][R][K]. Ranks that fill up R have no inputs:
// theirs is the adapter's first row, of which nothing is read.
constexpr long long rank_at(int a, int rank, int R, int K) {
  return ((long long)a * R + (rank < R ? rank : 0)) * K;
}

// Eight elements of 2 bytes from i on, of which those below `end` count, are read as words of 4 bytes: whether word j (of
// five) is. odd: element i is the second one of word 0. The word that has element i - 1 beside i is wanted only if i counts.
constexpr bool word_wanted(int i, int j, int odd, int end) { return i < end && i + 2 * j - odd < end && (j < 4 || odd); }

}  // namespace ds
