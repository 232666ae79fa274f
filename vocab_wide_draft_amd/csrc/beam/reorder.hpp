// Reordering of the beams' states (dspark_beam_reorder): every slot of a
// request takes the state of its parent.
//
// A thread owns one or two vectors of every beam of a request: it loads what
// the slots take, all of it on its way at once, and only then stores, so that
// states can be reordered in place without a second copy and without waiting
// for other threads.  A parent is loaded once however many slots take it, and
// what a slot keeps is neither read nor written.  Memory bounds it: 32 requests
// of eight beams, four states of up to 2,048 positions of 2 KB, move 5.07 GB
// into other states in 1,070 us (4.7 TB/s, a copy's rate), 2.34 GB in place in
// 460 us; with one vector a thread 1,590 and 970 us.  More beams leave fewer waves
// a SIMD (registers for a vector of each), and from 17 beams on vectors of 8 or 4
// bytes: two states of 2,048 positions of 2 KB, 256 beams in all, in place / into
// others, TB/s: 4 beams a request 5.7 / 5.3, 8 5.2 / 4.8, 12 4.0 / 4.3, 16 4.3 / 4.1,
// 32 4.5 / 3.9, 64 3.7 / 4.2.
#pragma once
#include "../logits/slices.hpp"

namespace dspark {

constexpr int kStates = 16;  // states of one launch

struct ReorderState {
  const char* in;
  char* out;
  int64_t in_request, in_beam, in_outer, in_row;      // strides in bytes
  int64_t out_request, out_beam, out_outer, out_row;
  int64_t row_bytes;
  int64_t rows, outer;         // rows: 0 for a state without positions, which is one row
  uint32_t vectors, chunks;    // of a row; workgroups of the longest stretch
  bool flat;                   // rows lie next to each other
};
struct ReorderArgs {
  ReorderState state[kStates];
  int64_t first[kStates + 1];  // workgroups before each state's
  int n_states, beams;
  int64_t requests;
  const int32_t* parent;
  const int32_t* length;
  int32_t* status;
  int64_t least_rows;  // positions that every state has
  bool in_place;
};

template <int N>
struct Size { static constexpr int value = N; };

// BYTES bytes at any address
template <int BYTES>
struct Word;
template <>
struct Word<16> { typedef v4u T __attribute__((aligned(1))); };
template <>
struct Word<8> { typedef v2u T __attribute__((aligned(1))); };
template <>
struct Word<4> { typedef uint32_t T __attribute__((aligned(1))); };
template <>
struct Word<2> { typedef uint16_t T __attribute__((aligned(1))); };
template <>
struct Word<1> { typedef uint8_t T; };

// PER vectors of a thread (those that are `on`); takes: the slots by parent.
template <int BYTES, int NB, int PER>
__device__ __forceinline__ void reorder_move(const ReorderState& st, const char* const (&in)[PER], char* const (&out)[PER], const bool (&on)[PER],
                                             const uint64_t (&takes)[NB]) {
  typedef typename Word<BYTES>::T W;
  W w[PER][NB];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (takes[b] && on[i]) w[i][b] = *reinterpret_cast<const W*>(in[i] + b * st.in_beam);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      for (uint64_t left = takes[b]; left; left &= left - 1)
        if (on[i]) *reinterpret_cast<W*>(out[i] + __builtin_ctzll(left) * st.out_beam) = w[i][b];
    }
  }
}

template <int BYTES, int NB, int PER>
__global__ void __launch_bounds__(kSliceBS) reorder_kernel(ReorderArgs a) {
  const int64_t block = block_number(a.first[a.n_states]);
  if (block < 0) return;
  int k = 0;
  while (block >= a.first[k + 1]) ++k;  // (uniform)
  const ReorderState& st = a.state[k];
  int64_t unit = block - a.first[k];
  const uint32_t chunk = (uint32_t)((uint64_t)unit % st.chunks);
  unit = (int64_t)((uint64_t)unit / st.chunks);
  const int64_t o = unit % st.outer, r = unit / st.outer;
  // every workgroup of a request finds the same faults
  const int lane = lane_id();
  const int32_t p = lane < a.beams ? a.parent[r * a.beams + lane] : -1;
  const int64_t len = a.length ? a.length[r] : st.rows;
  const bool bad_parent = __ballot(p < -1 || p >= a.beams) != 0, bad_length = a.length && (len < 0 || len > a.least_rows);
  if (k == 0 && o == 0 && chunk == 0) {
    if (threadIdx.x == 0 && a.status)
      a.status[r] = bad_parent ? DSPARK_ST_BAD_PARENT : bad_length ? DSPARK_ST_BAD_LENGTH : DSPARK_ST_OK;
  }
  if (bad_parent || bad_length) return;
  const bool moves = p >= 0 && !(a.in_place && p == lane);
  uint64_t takes[NB];  // the slots that take a parent's state
#pragma unroll
  for (int b = 0; b < NB; ++b) takes[b] = __ballot(moves && p == b);
  const char* in = st.in + r * st.in_request + o * st.in_outer;
  char* out = st.out + r * st.out_request + o * st.out_outer;
  const int64_t rows = st.rows ? len : 1;
  const int64_t total = st.flat ? rows * st.row_bytes / BYTES : rows * st.vectors;  // whole vectors, or those of a row with its rest
  const int64_t v0 = (int64_t)chunk * (kSliceBS * PER) + threadIdx.x;
  const char* from[PER];
  char* to[PER];
  bool on[PER];
  int rest = 0;  // bytes behind the whole vectors: of a row, or of the stretch
  const char* rest_from = nullptr;
  char* rest_to = nullptr;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t v = v0 + i * kSliceBS;
    on[i] = v < total;
    if (st.flat) {
      from[i] = in + v * BYTES;
      to[i] = out + v * BYTES;
      if (v == total) {
        rest = (int)(rows * st.row_bytes - total * BYTES);
        rest_from = from[i];
        rest_to = to[i];
      }
    } else {
      const int64_t row = (int64_t)((uint64_t)v / st.vectors);
      const int64_t col = (v - row * st.vectors) * BYTES;
      from[i] = in + row * st.in_row + col;
      to[i] = out + row * st.out_row + col;
      if (on[i] && col + BYTES > st.row_bytes) {
        on[i] = false;
        if constexpr (PER == 1) {
          rest = (int)(st.row_bytes - col);
          rest_from = from[i];
          rest_to = to[i];
        }
      }
    }
  }
  reorder_move<BYTES, NB, PER>(st, from, to, on, takes);
  if (rest) {
    int at = 0;
    const auto piece = [&](auto size) {
      constexpr int S = decltype(size)::value;
      if constexpr (S < BYTES) {
        if (rest & S) {
          const char* const f[1] = {rest_from + at};
          char* const t[1] = {rest_to + at};
          const bool yes[1] = {true};
          reorder_move<S, NB, 1>(st, f, t, yes, takes);
          at += S;
        }
      }
    };
    piece(Size<8>{});
    piece(Size<4>{});
    piece(Size<2>{});
    piece(Size<1>{});
  }
}

}  // namespace dspark
