// Reordering of the beams' states (dspark_beam_reorder): every slot of a
// request takes the state of its parent.
//
// A thread owns one vector of every beam of a request: it loads what each
// slot takes, all of them on their way at once, and only then stores, so that
// states can be reordered in place without a second copy and without waiting
// for other threads.  What a slot keeps is neither read nor written.
#pragma once
#include "../logits/slices.hpp"

namespace dspark {

constexpr int kStates = 16;  // states of one launch

struct ReorderState {
  const char* in;
  char* out;
  int64_t in_request, in_beam, in_outer, in_row;      // strides in bytes
  int64_t out_request, out_beam, out_outer, out_row;
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

template <int BYTES>
struct Word;
template <>
struct Word<16> { typedef v4u T; };
template <>
struct Word<8> { typedef v2u T; };
template <>
struct Word<4> { typedef uint32_t T; };
template <>
struct Word<2> { typedef uint16_t T; };
template <>
struct Word<1> { typedef uint8_t T; };

template <int BYTES, int NB>
__global__ void __launch_bounds__(kSliceBS) reorder_kernel(ReorderArgs a) {
  typedef typename Word<BYTES>::T W;
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
  const int32_t* parent = a.parent + r * a.beams;
  const int lane = lane_id();
  const int32_t p = lane < a.beams ? parent[lane] : -1;
  const int64_t len = a.length ? a.length[r] : st.rows;
  const bool bad_parent = __ballot(p < -1 || p >= a.beams) != 0, bad_length = a.length && (len < 0 || len > a.least_rows);
  if (k == 0 && o == 0 && chunk == 0) {
    if (threadIdx.x == 0 && a.status)
      a.status[r] = bad_parent ? DSPARK_ST_BAD_PARENT : bad_length ? DSPARK_ST_BAD_LENGTH : DSPARK_ST_OK;
  }
  if (bad_parent || bad_length) return;
  const uint64_t moves = __ballot(p >= 0 && !(a.in_place && p == lane));
  const int64_t v = (int64_t)chunk * kSliceBS + threadIdx.x;
  if (v >= (st.rows ? len : 1) * st.vectors) return;
  int64_t from = v * BYTES, to = from;
  if (!st.flat) {
    const int64_t row = (int64_t)((uint64_t)v / st.vectors), col = (v - row * st.vectors) * BYTES;
    from = row * st.in_row + col;
    to = row * st.out_row + col;
  }
  const char* in = st.in + r * st.in_request + o * st.in_outer + from;
  char* out = st.out + r * st.out_request + o * st.out_outer + to;
  W w[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (moves >> b & 1ull) w[b] = *reinterpret_cast<const W*>(in + (int64_t)parent[b] * st.in_beam);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (moves >> b & 1ull) *reinterpret_cast<W*>(out + b * st.out_beam) = w[b];
  }
}

}  // namespace dspark
