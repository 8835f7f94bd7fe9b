// Host side of what follows a product (ends.hpp): checks of the arguments, and which launch a choice stands for.
#pragma once

#include <initializer_list>

#include "block128_choose.hpp"
#include "block128_launch.hpp"
#include "host_checks.hpp"
#include "overlap.hpp"

namespace mxg {
namespace b128 {

// Types and distances between rows; those of a tensor that is not there do not matter.
inline int check_ends(const mxgemm_ends_t& e, int64_t N, int c_dtype) {
  if (e.activation < MXG_ACT_NONE || e.activation > MXG_ACT_GELU_TANH) return MXG_ERR_FMT;
  if (e.bias && e.bias_dtype != c_dtype && e.bias_dtype != MXG_DT_F32) return MXG_ERR_FMT;
  const struct {
    const void* at;
    int64_t ld;
  } all[] = {{e.gate, e.ldgate}, {e.residual, e.ldresidual}, {e.preact, e.ldpreact}};
  // as C's, and a tile's rows are addressed with 32-bit byte offsets
  for (const auto& t : all)
    if (t.at && (t.ld < N || t.ld > (1LL << 21))) return MXG_ERR_SHAPE;
  return MXG_OK;
}

inline bool ends_aligned(const mxgemm_ends_t& e, int c_dtype) {
  const size_t n = elem_bytes(c_dtype);
  return host::aligned_to(e.bias, elem_bytes(e.bias && e.bias_dtype == MXG_DT_F32 ? MXG_DT_F32 : c_dtype)) &&
         host::aligned_to(e.gate, n) && host::aligned_to(e.residual, n) && host::aligned_to(e.preact, n);
}

inline bool ends_on_device(const mxgemm_ends_t& e, int dev) {
  for (const void* t : {e.bias, e.gate, e.residual, (const void*)e.preact})
    if (t && !host::on_device(t, dev)) return false;
  return true;
}

// Whether an output lies on anything that the call reads or writes besides: workgroups would read what others have written.
// Only gate and residual may be C, the same rows of it, which the lanes that write them have read before.
inline bool outputs_overlap(const host::RowsAt& c, const mxgemm_ends_t* e, int c_dtype, std::initializer_list<host::RowsAt> others) {
  using namespace host;
  for (const RowsAt& o : others)
    if (overlap(c, o)) return true;
  if (!e) return false;
  const int64_t n = elem_bytes(c_dtype), N = c.bytes / n;
  const RowsAt bias = flat(e->bias, N * elem_bytes(e->bias_dtype)), gate = rows_at(e->gate, c.rows, N, e->ldgate, n),
               residual = rows_at(e->residual, c.rows, N, e->ldresidual, n), z = rows_at(e->preact, c.rows, N, e->ldpreact, n);
  for (const RowsAt& o : others)
    if (overlap(z, o)) return true;
  for (const RowsAt& o : {gate, residual})
    if (overlap(z, o) || (overlap(c, o) && !same(c, o))) return true;
  return overlap(c, bias) || overlap(z, bias) || overlap(c, z);
}

// Whether rows of all tensors beside C are whole 16-byte chunks, `per` elements each.
inline bool ends_whole(const mxgemm_ends_t& e, int per) {
  return (!e.gate || (host::aligned16(e.gate) && e.ldgate % per == 0)) &&
         (!e.residual || (host::aligned16(e.residual) && e.ldresidual % per == 0)) &&
         (!e.preact || (host::aligned16(e.preact) && e.ldpreact % per == 0));
}

inline ends::Ends kernel_ends(const mxgemm_ends_t& e) {
  ends::Ends k{};
  k.bias = e.bias;
  k.gate = e.gate;
  k.residual = e.residual;
  k.Z = e.preact;
  k.ldg = e.ldgate;
  k.ldr = e.ldresidual;
  k.ldz = e.ldpreact;
  k.act = e.activation;
  k.bias_f32 = e.bias_dtype == MXG_DT_F32;
  return k;
}

inline TileLaunch tile_launch(const Choice& c, bool exact) {
  if (exact) return c.bn == 256 ? launch_exact128x256 : c.bm == 128 ? launch_exact128 : c.bn == 128 ? launch_exact64x128 : launch_exact64;
  return c.bm == 256   ? launch_tile256
         : c.bn == 256 ? launch_tile128x256
         : c.bm == 128 ? launch_tile128
         : c.bn == 128 ? launch_tile64x128
                       : launch_tile64;
}

inline MoreLaunch more_launch(const Choice& c, bool exact) {
  if (exact)
    return c.bn == 256 ? launch_more_exact128x256 : c.bm == 128 ? launch_more_exact128 : c.bn == 128 ? launch_more_exact64x128 : launch_more_exact64;
  return c.bm == 256   ? launch_more256
         : c.bn == 256 ? launch_more128x256
         : c.bm == 128 ? launch_more128
         : c.bn == 128 ? launch_more64x128
                       : launch_more64;
}

}  // namespace b128
}  // namespace mxg
