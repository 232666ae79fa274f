// Beam search on logit rows: the selection over beams and vocabulary, and the
// reordering of the beams' states (the entry points declared in
// include/dspark.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <memory>
#include <new>

#include "../host_checks.hpp"
#include "dspark.h"
#include "regions.hpp"
#include "reorder.hpp"
#include "select.hpp"

namespace dspark {
namespace {

static_assert(kBeams == DSPARK_BEAM_MAX && kBeamOut == DSPARK_BEAM_OUT_MAX, "limits of the interface");

struct BeamPlan {
  int slice, slices, cap;
  size_t part_at, bytes;
};
BeamPlan beam_plan_of(int64_t n, int64_t V, int n_out, int slice) {
  BeamPlan p{};
  p.slice = slice;
  p.slices = (int)((V + slice - 1) / slice);
  p.cap = beam_cap(n_out);
  p.part_at = (size_t)n * (size_t)p.slices * (size_t)p.cap * sizeof(uint64_t);
  p.bytes = p.part_at + (size_t)n * (size_t)p.slices * sizeof(BeamPart);
  return p;
}
// The most logits of a slice: 8,192, or fewer where those leave CUs idle and
// the join takes as many slices.
constexpr int64_t kBeamWant = 512;
int beam_slice(int64_t n, int64_t V) {
  int slice = 8192;
  while (slice > 2048 && n * ((V + slice - 1) / slice) < kBeamWant && V <= (int64_t)slice / 2 * kBeamSlices) slice /= 2;
  return slice;
}
BeamPlan beam_plan(int64_t n, int64_t V, int n_out) { return beam_plan_of(n, V, n_out, beam_slice(n, V)); }

template <int DT>
void launch_select(const BeamArgs& a, int slice, hipStream_t s) {
  constexpr int step = kSliceBS * kVec<DT>;
  const dim3 grid = row_slice_grid(a.x.n, a.slices);
  if (slice == 2048) hipLaunchKernelGGL(HIP_KERNEL_NAME(beam_slice_kernel<DT, 2048 / step>), grid, dim3(kSliceBS), 0, s, a);
  else if (slice == 4096) hipLaunchKernelGGL(HIP_KERNEL_NAME(beam_slice_kernel<DT, 4096 / step>), grid, dim3(kSliceBS), 0, s, a);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(beam_slice_kernel<DT, 8192 / step>), grid, dim3(kSliceBS), 0, s, a);
  hipLaunchKernelGGL(HIP_KERNEL_NAME(beam_join_kernel<DT, 8>), grid_of(a.requests), dim3(512),
                     beam_join_bytes(a.beams, a.slices, a.n_out, 8), s, a);
}

// the bytes that a state's layout spans; -1 where parts overlap, or it is longer than any memory
int64_t span(const int64_t (&size)[4], const int64_t (&stride)[4], int64_t row_bytes, bool apart) {
  int order[4] = {0, 1, 2, 3};
  std::sort(order, order + 4, [&](int a, int b) { return stride[a] < stride[b]; });
  int64_t reach = row_bytes;
  for (int i : order) {
    if (size[i] <= 1) continue;
    if (stride[i] < 0 || (apart && stride[i] < reach) || stride[i] > (int64_t(1) << 56) / size[i]) return -1;
    reach += stride[i] * (size[i] - 1);
  }
  return reach;
}

template <int BYTES, int NB>
void launch_reorder(const ReorderArgs& a, int per, hipStream_t s) {
  const dim3 grid = grid_of(a.first[a.n_states]);
  if (per == 2) hipLaunchKernelGGL(HIP_KERNEL_NAME(reorder_kernel<BYTES, NB, 2>), grid, dim3(kSliceBS), 0, s, a);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(reorder_kernel<BYTES, NB, 1>), grid, dim3(kSliceBS), 0, s, a);
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

size_t dspark_beam_select_workspace(int64_t n_rows, int64_t vocab, int32_t n_out) {
  if (n_rows <= 0 || n_rows > (1 << 24) || vocab < 1 || vocab > DSPARK_V_MAX || n_out < 1 || n_out > DSPARK_BEAM_OUT_MAX) return 0;
  // fewer rows may have more slices: the most rows that have slices of each length
  size_t bytes = beam_plan(n_rows, vocab, n_out).bytes;
  for (int64_t slice = 4096; slice <= 8192; slice *= 2) {
    const int64_t rows = std::min<int64_t>(n_rows, (kBeamWant - 1) / ((vocab + slice - 1) / slice));
    if (rows > 0) bytes = std::max(bytes, beam_plan(rows, vocab, n_out).bytes);
  }
  return bytes;
}

int dspark_beam_select(const dspark_rows* rows, const float* scores, const int32_t* finished, int32_t beams,
                       int32_t n_out, int32_t end_token, int32_t* parent, int32_t* token, float* score,
                       int32_t* out_finished, int32_t* len, int32_t* req_status, void* ws, size_t ws_bytes,
                       void* stream) {
  int rc = host_check_rows(rows, "rows NULL");
  if (rc) return rc;
  if (beams < 1 || beams > DSPARK_BEAM_MAX) return fail(DSPARK_EINVAL, "beams must be in [1, DSPARK_BEAM_MAX]");
  if (n_out < 1 || n_out > DSPARK_BEAM_OUT_MAX) return fail(DSPARK_EINVAL, "n_out must be in [1, DSPARK_BEAM_OUT_MAX]");
  if (beams * n_out > 4096) return fail(DSPARK_EINVAL, "beams * n_out must be at most 4096");
  if (rows->n_rows % beams != 0) return fail(DSPARK_EINVAL, "n_rows is not a multiple of beams");
  if (end_token < -1 || end_token >= rows->vocab) return fail(DSPARK_EINVAL, "end_token must be in [-1, vocab)");
  if (finished && end_token < 0) return fail(DSPARK_EINVAL, "finished needs an end_token");
  if (rows->n_rows == 0) return DSPARK_SUCCESS;
  if (!scores || !parent || !token || !score || !out_finished || !len || !req_status) return fail(DSPARK_EINVAL, "NULL scores or output");
  const BeamPlan p = beam_plan(rows->n_rows, rows->vocab, n_out);
  if (!aligned16(ws)) return fail(DSPARK_EALIGN, "workspace must be 16-byte aligned");
  if (!ws || ws_bytes < p.bytes) return fail(DSPARK_EWORKSPACE, "workspace smaller than dspark_beam_select_workspace()");
  const int64_t requests = rows->n_rows / beams, all = requests * n_out * 4, es = rows->dtype == DSPARK_BF16 ? 2 : 4;
  const int64_t row_count[4] = {rows->n_rows, 1, 1, 1}, row_step[4] = {rows->row_stride * es, 0, 0, 0};
  Region region[] = {region_of(rows->data, row_count, row_step, rows->vocab * es, 0, false),
                     piece_of(scores, rows->n_rows * 4, 1, false), piece_of(finished, rows->n_rows * 4, 2, false),
                     piece_of(parent, all, 3, true), piece_of(token, all, 4, true), piece_of(score, all, 5, true),
                     piece_of(out_finished, all, 6, true), piece_of(len, requests * 4, 7, true),
                     piece_of(req_status, requests * 4, 8, true), piece_of(ws, (int64_t)p.bytes, 9, true)};
  if (any_meet(region, sizeof region / sizeof *region)) return fail(DSPARK_EINVAL, "an output or the workspace overlaps an input or another output");
  BeamArgs a{};
  a.x.n = rows->n_rows;
  a.x.x = rows->data;
  a.x.stride = rows->row_stride;
  a.x.V = (int)rows->vocab;
  a.x.inv_t = 1.0;
  a.x.c = (float)1.4426950408889634;
  a.scores = scores;
  a.finished = finished;
  a.beams = beams;
  a.n_out = n_out;
  a.end_token = end_token;
  a.requests = requests;
  a.parent = parent;
  a.token = token;
  a.score = score;
  a.out_finished = out_finished;
  a.len = len;
  a.status = req_status;
  a.slices = p.slices;
  a.length = (int)((rows->vocab + p.slices * 8 - 1) / (p.slices * 8) * 8);
  a.cap = p.cap;
  a.cand = static_cast<uint64_t*>(ws);
  a.part = reinterpret_cast<BeamPart*>(static_cast<char*>(ws) + p.part_at);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows->dtype == DSPARK_F32) launch_select<DSPARK_F32>(a, p.slice, s);
  else launch_select<DSPARK_BF16>(a, p.slice, s);
  return host_check_launch();
}

int dspark_beam_reorder(const dspark_state* states, int32_t n_states, int64_t requests, int32_t beams,
                        const int32_t* parent, const int32_t* length, int32_t* req_status, void* stream) {
  if (n_states < 1 || !states) return fail(DSPARK_EINVAL, "no states");
  if (requests < 0 || requests > (1 << 24)) return fail(DSPARK_EINVAL, "requests out of range");
  if (beams < 1 || beams > DSPARK_BEAM_MAX) return fail(DSPARK_EINVAL, "beams must be in [1, DSPARK_BEAM_MAX]");
  const bool in_place = states[0].in == states[0].out;
  int64_t least = INT64_MAX;
  // what the call reads and writes
  constexpr int kFew = 64;
  Region few[kFew];
  const int64_t pieces = (in_place ? 1 : 2) * (int64_t)n_states + 3;
  std::unique_ptr<Region[]> many(pieces > kFew ? new (std::nothrow) Region[pieces] : nullptr);
  Region* const region = pieces > kFew ? many.get() : few;
  if (!region) return fail(DSPARK_EINVAL, "too many states for the host's memory");
  int n_regions = 0;
  if (requests > 0) {
    region[n_regions++] = piece_of(parent, requests * beams * 4, -1, false);
    region[n_regions++] = piece_of(length, requests * 4, -2, false);
    region[n_regions++] = piece_of(req_status, requests * 4, -3, true);
  }
  for (int i = 0; i < n_states; ++i) {
    const dspark_state& t = states[i];
    if (t.outer < 1 || t.rows < 0 || t.row_bytes < 1 || t.row_bytes > INT32_MAX || t.outer > (1 << 24) || t.rows > INT32_MAX ||
        t.rows * t.row_bytes >= (int64_t(1) << 39))
      return fail(DSPARK_EINVAL, "a state's outer, rows or row_bytes is out of range");
    const int64_t size[4] = {requests, beams, t.outer, std::max<int64_t>(t.rows, 1)};
    const int64_t in[4] = {t.in_request, t.in_beam, t.in_outer, t.in_row}, out[4] = {t.out_request, t.out_beam, t.out_outer, t.out_row};
    const int64_t in_span = span(size, in, t.row_bytes, false), out_span = span(size, out, t.row_bytes, true);
    if (in_span < 0 || out_span < 0) return fail(DSPARK_EINVAL, "a state's strides make its parts overlap");
    if (requests > 0 && (!t.in || !t.out)) return fail(DSPARK_EINVAL, "NULL state");
    if ((t.in == t.out) != in_place) return fail(DSPARK_EINVAL, "all states must be in place, or none");
    for (int d = 0; d < 4; ++d) {
      if (size[d] <= 1) continue;
      if (in_place && in[d] != out[d]) return fail(DSPARK_EINVAL, "in place needs the same strides");
    }
    if (!in_place) {
      const char *x = static_cast<const char*>(t.in), *y = static_cast<const char*>(t.out);
      if (x < y + out_span && y < x + in_span) return fail(DSPARK_EINVAL, "a state's output overlaps its input");
    }
    if (requests > 0) {
      region[n_regions++] = region_of(t.out, size, out, t.row_bytes, i, true);
      if (!in_place) region[n_regions++] = region_of(t.in, size, in, t.row_bytes, i, false);
    }
    if (t.rows > 0) least = std::min(least, t.rows);
  }
  if (any_meet(region, n_regions)) return fail(DSPARK_EINVAL, "a state, parent, length or req_status overlaps another one that is written");
  if (requests == 0) return DSPARK_SUCCESS;
  if (!parent || !req_status) return fail(DSPARK_EINVAL, "NULL parent or req_status");
  // 16 bytes of every beam to a thread, fewer where that would be too many registers
  const int bytes = beams <= 16 ? 16 : beams <= 32 ? 8 : 4;
  hipStream_t s = static_cast<hipStream_t>(stream);
  for (int at = 0; at < n_states; at += kStates) {
    ReorderArgs a{};
    a.n_states = std::min(kStates, n_states - at);
    a.beams = beams;
    a.requests = requests;
    a.parent = parent;
    a.length = length;
    a.status = at == 0 ? req_status : nullptr;
    a.least_rows = least == INT64_MAX ? INT32_MAX : least;
    a.in_place = in_place;
    bool flat = true;
    int64_t vectors = 0;
    for (int i = 0; i < a.n_states; ++i) {
      const dspark_state& t = states[at + i];
      ReorderState& u = a.state[i];
      u.in = static_cast<const char*>(t.in);
      u.out = static_cast<char*>(t.out);
      u.in_request = t.in_request;
      u.in_beam = t.in_beam;
      u.in_outer = t.in_outer;
      u.in_row = t.in_row;
      u.out_request = t.out_request;
      u.out_beam = t.out_beam;
      u.out_outer = t.out_outer;
      u.out_row = t.out_row;
      u.row_bytes = t.row_bytes;
      u.rows = t.rows;
      u.outer = t.outer;
      u.flat = t.rows <= 1 || (t.in_row == t.row_bytes && t.out_row == t.row_bytes);
      u.vectors = (uint32_t)((t.row_bytes + bytes - 1) / bytes);
      flat = flat && (u.flat || t.row_bytes % bytes == 0);
      vectors += requests * t.outer * std::max<int64_t>(t.rows, 1) * (int64_t)u.vectors;
    }
    // two vectors of every beam on their way to a thread, where the states are large and their rows hold whole vectors
    const int per = !flat || vectors < (1 << 20) ? 1 : 2;
    for (int i = 0; i < a.n_states; ++i) {
      ReorderState& u = a.state[i];
      const int64_t rows = std::max<int64_t>(u.rows, 1);
      // (a flat stretch has one vector more for what is left behind the whole ones)
      const int64_t all = u.flat ? rows * u.row_bytes / bytes + 1 : rows * (int64_t)u.vectors;
      u.chunks = (uint32_t)((all + kSliceBS * per - 1) / (kSliceBS * per));
      a.first[i + 1] = a.first[i] + requests * u.outer * (int64_t)u.chunks;
    }
    if (beams <= 4) launch_reorder<16, 4>(a, per, s);
    else if (beams <= 8) launch_reorder<16, 8>(a, per, s);
    else if (beams <= 16) launch_reorder<16, 16>(a, per, s);
    else if (beams <= 32) launch_reorder<8, 32>(a, per, s);
    else launch_reorder<4, 64>(a, per, s);
  }
  return host_check_launch();
}

}  // extern "C"
