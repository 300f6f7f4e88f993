// Host-only checks and workspace layout of the mixture-of-experts layer.
#include <stdint.h>

#include "../../include/mm.h"
#include "plan.h"

namespace qsg {

namespace {

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace

int make_moe_plan(int type, int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k, MoePlan* p) {
  *p = MoePlan();
  if (type != MM_TYPE_Q4_0R && type != MM_TYPE_F8 && type != MM_TYPE_F16) return MM_ERR_ARG;
  if (T < 0 || T > kMoeMaxTokens || D < 1 || D > kMoeMaxDim || D % kQK || F < 1 || F > kMoeMaxDim ||
      F % kQK || E < 1 || E > kMoeMaxExperts || top_k < 1 || top_k > kMoeMaxTopK || top_k > E)
    return MM_ERR_SHAPE;
  if (T == 0) return MM_OK;
  size_t off = 0;
  const auto take = [&off](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  const size_t slots = (size_t)(T * top_k);
  p->off_logits = take((size_t)(T * E) * 8);
  p->off_ids = take(slots * 4);
  p->off_weights = take(slots * 4);
  p->off_xp = take((size_t)(T * D) * 4);
  p->off_xs = take((size_t)T * align_up((size_t)(D / kQK), 4) * 4);
  p->off_hp = take(slots * (size_t)F * 4);
  p->off_hs = take(slots * align_up((size_t)(F / kQK), 4) * 4);
  // The selection costs each workgroup of the next launch about T E^2 / 512
  // steps per thread where it makes it itself.
  p->fold = T * E * E <= 65536;
  // Down: 16 rows per workgroup while an expert serves few tokens; with more,
  // 64 rows share each activation load (activations are 4 bytes a value, the
  // weights as few as half a byte) and the sequence of (expert, unit) pairs
  // is cut in slices to fill the device.
  const int64_t used = T * top_k < E ? T * top_k : E;
  // Gate / up: groups of 32 rows, several per workgroup where that leaves a grid of
  // two workgroups per CU if every expert that can be in use is.  Registers or LDS
  // let one run on a CU at a time; the second is there for calls that use fewer
  // experts than they could (whole layer, us, grids of about 3 / 2 / 1 per CU, 8
  // experts of 4096 x 14336, Q4_0R: 32 tokens 246 / 232 / 229, 16 tokens 221 / 203 /
  // 199; 4 tokens on 7 of the experts 179 / 166 / 163, on 3 or 4 of them 98 / 94 / 134).
  const int64_t groups = F / kQK, per = groups * used / (2 * kCUs);
  p->up_groups = (int)(per > 1 ? (groups + per - 1) / per : groups);
  const bool many = T * top_k > 2 * used;
  const bool few = T <= kMoeFewTokens;
  // (the per-wave sums of T tokens x 16 rt rows, 8 waves, share the LDS with
  // the staging, which e4m3 weights need too)
  const bool f8 = type == MM_TYPE_F8;
  p->rt = few || !many ? 1 : !f8 && D % 64 == 0 && T <= 32 ? 4 : D % 32 == 0 && T <= (f8 ? 32 : 64) ? 2 : 1;
  const int64_t tiles = D / (16 * p->rt), units = used * ((F / kQK + 3) / 4);
  int64_t slices = few ? 1 : p->rt > 1 ? (2 * kCUs + tiles - 1) / tiles : kCUs / tiles;
  if (slices > units / 64) slices = units / 64;
  p->slices = (int)(slices < 1 ? 1 : slices > 8 ? 8 : slices);
  if (p->slices > 1) p->off_part = take((size_t)p->slices * (size_t)(T * D) * 4);
  p->ws_bytes = off;
  return MM_OK;
}

}  // namespace qsg
