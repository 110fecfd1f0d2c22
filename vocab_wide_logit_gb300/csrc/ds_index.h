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
// Chunks that hold a row of V.
constexpr unsigned chunks_of(int V, int E, int dc) { return ((unsigned)V + dc + E - 1) / E; }
// The number of a chunk's first logit, below 0 in front of a row that starts within a chunk. Of a chunk that the row has.
constexpr int first_of_chunk(unsigned chunk, int E, int dc) { return (int)(chunk * E - dc); }
// Whether logit i of the chunk whose first one is number `first` is the row's, and whether all E of them are.
constexpr bool in_row(int first, int i, int V) { return (unsigned)first + i < (unsigned)V; }
constexpr bool all_in_row(int first, int E, int V) { return first >= 0 && V - first >= E; }
// Where the token is among the logits from number `first` on: below E if it is in that chunk. Of a token >= 0.
constexpr unsigned place_of(int token, int first) { return (unsigned)token - (unsigned)first; }

}  // namespace ds
