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

// ---------------------------------------------------------------- a row's chunks of 16 bytes
// Of E logits each, the first of which has dc that are before the row. A row may have 2^31 - 1 logits: a sum of a logit's
// number and a place in a chunk passes 32 bits.
// The chunk that has logit `id`.
constexpr int chunk_of(int id, int E, int dc) { return (int)(((long long)id + dc) / E); }
// The first logit of the row in a chunk that has one.
constexpr int first_in_chunk(int chunk, int E, int dc) {
  const long long id = (long long)chunk * E - dc;
  return id < 0 ? 0 : (int)id;
}
// Whether the logit `place` behind the first one of the token's chunk is in front of the token (-1, in chunk 0: none is).
constexpr bool in_front_of(int token, int first, int place) { return place < token - first; }

}  // namespace ds
