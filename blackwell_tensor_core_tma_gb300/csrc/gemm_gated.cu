// Instances of the gated product's kernels (gemm_gated.cuh):
//   forward, 16-bit    pairs of CTAs, 256 x (128 + 128) tiles, 6 stages; single CTAs, 128 x (64 + 64) tiles, whole
//                      or sliced along K
//   forward, e4m3      the same tiles; a pair's accumulator takes half of tensor memory and the scales of
//                      the stages part of the rest, so that the epilogue empties it into registers at once
//   backward, 16-bit   pairs, 256 x 256 tiles; single CTAs, 128 x 128 and 128 x 64 tiles, whole or sliced
// each with as many stages as shared memory holds.
#include "gemm_gated.cuh"

namespace gb300 {
namespace {

using F16Pair = GatedInstance<GatedCfg<2, KIND_F16, false, 128, 6, 2, 8>>;
using F16Single = GatedInstance<GatedCfg<1, KIND_F16, false, 64, 6, 2, 8, 0, false, false, 2>>;
using F16Sliced = GatedInstance<GatedCfg<1, KIND_F16, false, 64, 5, 2, 8, 0, false, true>>;
using Mx8Pair = GatedInstance<GatedCfg<2, KIND_MXF8, false, 128, 5, 1, 8, 2>>;
using Mx8Single = GatedInstance<GatedCfg<1, KIND_MXF8, false, 64, 5, 2, 8, 2, true>>;
using Mx8SinglePacked = GatedInstance<GatedCfg<1, KIND_MXF8, false, 64, 5, 2, 8, 1>>;
using Mx8Sliced = GatedInstance<GatedCfg<1, KIND_MXF8, false, 64, 4, 2, 8, 2, true, true>>;
using Mx8SlicedPacked = GatedInstance<GatedCfg<1, KIND_MXF8, false, 64, 4, 2, 8, 1, false, true>>;
using BackPair = GatedInstance<GatedCfg<2, KIND_F16, true, 256, 5, 2, 8>>;
using BackSingle = GatedInstance<GatedCfg<1, KIND_F16, true, 128, 5, 2, 8, 0, false, false, 2>>;
using BackNarrow = GatedInstance<GatedCfg<1, KIND_F16, true, 64, 7, 2, 8, 0, false, false, 2>>;
using BackNarrowSliced = GatedInstance<GatedCfg<1, KIND_F16, true, 64, 7, 2, 8, 0, false, true, 2>>;
using BackSliced = GatedInstance<GatedCfg<1, KIND_F16, true, 128, 5, 2, 8, 0, false, true>>;

// f(instance) for a form, a CTA group and a number of slices
template <typename F>
auto with(GatedForm form, int cta_group, int slices, F f) {
    const bool pair = cta_group == 2, sliced = slices > 1;
    if (form == GATED_F16) return pair ? f(F16Pair()) : sliced ? f(F16Sliced()) : f(F16Single());
    if (form == GATED_MXF8) return sliced ? f(Mx8Sliced()) : f(Mx8Single());
    if (form == GATED_MXF8_PACKED) return pair ? f(Mx8Pair()) : sliced ? f(Mx8SlicedPacked()) : f(Mx8SinglePacked());
    if (form == GATED_BACK_NARROW) return sliced ? f(BackNarrowSliced()) : f(BackNarrow());
    return pair ? f(BackPair()) : sliced ? f(BackSliced()) : f(BackSingle());
}

}  // namespace

GatedShape gated_shape(GatedForm form, int cta_group, int slices) {
    return with(form, cta_group, slices, [](auto i) { return i.shape(); });
}
cudaError_t gated_prepare(GatedForm form, int cta_group, int slices, int *clusters) {
    return with(form, cta_group, slices, [&](auto i) { return i.prepare(slices, clusters); });
}
cudaError_t gated_launch(GatedForm form, int cta_group, int grid, const CUtensorMap *maps, const GatedParams &p,
                         cudaStream_t stream) {
    return with(form, cta_group, p.slices, [&](auto i) { return i.launch(grid, maps, p, stream); });
}

}  // namespace gb300
