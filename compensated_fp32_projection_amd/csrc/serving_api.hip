// C ABI of the rotary, 8-bit cache and beam calls (declared in
// include/cfp32.h): argument validation, the device check and workspace sizes.
// Every call validates all of its arguments before it enqueues anything.
#include "api_checks.h"
#include "rotary.h"

namespace {

using namespace cfp32;

// In place, or apart (which the caller sees to).
bool same_view(const void *in, int64_t s0, int64_t s1, const void *out, int64_t o0, int64_t o1)
{
    return in != out || (s0 == o0 && s1 == o1);
}

}  // namespace

extern "C" {

cfp32_status cfp32_rotary_frequencies(double theta, int64_t R, int scaling, double factor, double trained, double slow,
                                      double fast, double *frequencies, double *amplitude)
{
    if (!(theta > 0.0) || !std::isfinite(theta) || R < 2 || R % 2 || R > kRotaryMaxDim || !frequencies || !amplitude)
        return CFP32_ERR_INVALID_VALUE;
    if (scaling < CFP32_ROTARY_PLAIN || scaling > CFP32_ROTARY_PARTS) return CFP32_ERR_INVALID_VALUE;
    if (scaling != CFP32_ROTARY_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return CFP32_ERR_INVALID_VALUE;
    if (scaling == CFP32_ROTARY_PARTS &&
        !(trained > 0.0 && std::isfinite(trained) && std::isfinite(slow) && std::isfinite(fast) && slow < fast))
        return CFP32_ERR_INVALID_VALUE;
    const double n = (double)R;
    if (scaling == CFP32_ROTARY_NTK && R > 2) theta *= std::pow(factor, n / (n - 2.0));
    if (!std::isfinite(theta)) return CFP32_ERR_INVALID_VALUE;
    for (int64_t i = 0; i < R / 2; ++i) {
        double f = std::pow(theta, -2.0 * (double)i / n);
        if (scaling == CFP32_ROTARY_LINEAR) f /= factor;
        if (scaling == CFP32_ROTARY_PARTS) {
            const double turns = trained * f / 6.283185307179586476925286766559;
            const double g = std::fmin(std::fmax((turns - slow) / (fast - slow), 0.0), 1.0);
            f = g * f + (1.0 - g) * f / factor;
        }
        frequencies[i] = f;
    }
    *amplitude = scaling == CFP32_ROTARY_PARTS ? 1.0 + 0.1 * std::log(factor) : 1.0;
    return CFP32_OK;
}

cfp32_status cfp32_rotary(const void *q, int64_t q_tok, int64_t q_head, const void *k, int64_t k_tok, int64_t k_head, int type,
                          const int64_t *positions, const double *frequencies, double amplitude, int layout, int transpose,
                          void *q_out, int64_t qo_tok, int64_t qo_head, void *k_out, int64_t ko_tok, int64_t ko_head,
                          int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t R, void *stream)
{
    if (!size_ok(T) || !size_ok(Hq) || !size_ok(Hkv) || D < 0 || D > kRotaryMaxDim || R < 0 || R > D || R % 2 || !type_ok(type))
        return CFP32_ERR_INVALID_VALUE;
    if (Hq + Hkv > kMaxSize / kRotaryMaxDim) return CFP32_ERR_INVALID_VALUE;  // a token's items are counted in 32 bits
    if (layout != CFP32_ROTARY_HALF && layout != CFP32_ROTARY_INTERLEAVED) return CFP32_ERR_INVALID_VALUE;
    if (!scale_ok(amplitude)) return CFP32_ERR_INVALID_VALUE;
    if (T == 0 || D == 0 || Hq + Hkv == 0) return CFP32_OK;
    const size_t al = type == CFP32_KV_F16 ? 2 : 4;
    auto ok = [&](const void *in, int64_t s0, int64_t s1, const void *out, int64_t o0, int64_t o1, int64_t H) {
        return H == 0 || (in && out && aligned_to(in, al) && aligned_to(out, al) && view_ok(T, s0, H, s1, 1, 0, D) &&
                          view_ok(T, o0, H, o1, 1, 0, D) && distinct_ok(T, o0, H, o1, 1, 0, D) &&
                          same_view(in, s0, s1, out, o0, o1));
    };
    if (!ok(q, q_tok, q_head, q_out, qo_tok, qo_head, Hq) || !ok(k, k_tok, k_head, k_out, ko_tok, ko_head, Hkv))
        return CFP32_ERR_INVALID_VALUE;
    if ((R > 0 && !frequencies) || !aligned_to(frequencies, 8) || !aligned_to(positions, 8)) return CFP32_ERR_INVALID_VALUE;
    cfp32_status st = api_check_device();
    if (st != CFP32_OK) return st;
    const RotaryArgs a = {{q, q_out, q_tok, q_head, qo_tok, qo_head, (int)Hq}, {k, k_out, k_tok, k_head, ko_tok, ko_head, (int)Hkv},
                          positions, frequencies, (float)amplitude, type == CFP32_KV_F16, layout == CFP32_ROTARY_INTERLEAVED,
                          transpose != 0, (int)T, (int)D, (int)R};
    return api_launched(launch_rotary(a, (hipStream_t)stream));
}

}  // extern "C"
