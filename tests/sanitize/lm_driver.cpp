// Exercises the host side of the entry points around the mixer layer (argument
// checks, workspace sizing, empty problems) for a build whose host code runs
// under AddressSanitizer and UndefinedBehaviorSanitizer.  Every call returns
// before any device work.  Exit status 0 on success, 1 on an unexpected result.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "naju.h"

static int failures = 0;

static void expect(const char *what, naju_status_t got, naju_status_t want)
{
    const char *msg = naju_last_error();
    if (got != want || (got != NAJU_OK && std::strlen(msg) == 0)) {
        std::fprintf(stderr, "%s: status %d, expected %d (%s)\n", what, (int)got, (int)want, msg);
        ++failures;
    }
}

int main()
{
    alignas(256) static unsigned char buf[1 << 12];
    void *p = buf, *mis = buf + 1;
    int32_t *ip = (int32_t *)buf;
    float *fp = (float *)buf;
    const size_t big = (size_t)1 << 60;

    const int64_t Ts[] = {-1, 0, 1, 4095, 4096, 4097, (int64_t)1 << 28, ((int64_t)1 << 28) + 1,
                          INT64_MAX, INT64_MIN};
    const int64_t Vs[] = {-1, 0, 1, 511, 512, 100003, (int64_t)1 << 30, INT64_MAX};
    const int64_t ds[] = {-1, 0, 1, 768, (int64_t)1 << 20, INT64_MAX};
    for (int64_t T : Ts)
        for (int64_t V : Vs)
            for (int64_t d : ds) {
                (void)naju_embed_bwd_workspace_bytes(T, V, d);
                // no pointer: refused, or an empty problem
                naju_status_t s = naju_embed_fwd(T, V, d, NAJU_BF16, nullptr, nullptr, 1.f,
                                                 nullptr, nullptr);
                if (T > 0 && d > 0) expect("embed_fwd without pointers", s, NAJU_EINVAL);
                s = naju_embed_bwd(T, V, d, NAJU_F32, nullptr, nullptr, 1.f, 1, nullptr, nullptr,
                                   0, nullptr);
                if (V > 0 && d > 0) expect("embed_bwd without pointers", s, NAJU_EINVAL);
            }
    expect("embed_fwd io", naju_embed_fwd(1, 1, 1, 5, ip, p, 1.f, p, nullptr), NAJU_EINVAL);
    expect("embed_fwd alignment", naju_embed_fwd(1, 1, 1, NAJU_BF16, ip, mis, 1.f, p, nullptr),
           NAJU_EINVAL);
    expect("embed_bwd workspace",
           naju_embed_bwd(8, 8, 8, NAJU_BF16, ip, p, 1.f, 0, fp, p, 16, nullptr), NAJU_EWORKSPACE);
    expect("embed_bwd workspace alignment",
           naju_embed_bwd(8, 8, 8, NAJU_BF16, ip, p, 1.f, 0, fp, buf + 64, big, nullptr),
           NAJU_EINVAL);

    for (int64_t R : Ts)
        for (int64_t V : Vs)
            for (int64_t k : {(int64_t)-1, (int64_t)0, (int64_t)512, (int64_t)513, INT64_MAX}) {
                const naju_status_t s =
                    naju_distill_fwd(R, V, k, NAJU_F32, nullptr, V, nullptr, nullptr, 1.f, fp, fp,
                                     nullptr);
                if (R > 0 && V > 0 && s == NAJU_OK) {
                    std::fprintf(stderr, "distill_fwd without pointers accepted\n");
                    ++failures;
                }
            }
    expect("distill_bwd stride", naju_distill_bwd(2, 8, 1, NAJU_F32, p, 7, ip, fp, 1.f, fp, fp, p,
                                                  8, nullptr), NAJU_EINVAL);
    expect("distill_fwd_bwd temperature",
           naju_distill_fwd_bwd(2, 8, 1, NAJU_F32, p, 8, ip, fp, 0.f, fp, fp, fp, p, 8, nullptr),
           NAJU_EINVAL);

    for (int64_t R : Ts)
        for (int64_t V : Vs)
            for (int64_t n : {(int64_t)-1, (int64_t)0, (int64_t)4094, INT64_MAX}) {
                (void)naju_logits_workspace_bytes(R);
                const naju_status_t s = naju_logits_process(
                    R, V, NAJU_F32, nullptr, V, nullptr, n, nullptr, nullptr, nullptr, nullptr,
                    nullptr, nullptr, n, nullptr, nullptr, nullptr, nullptr, 0, nullptr);
                if (R > 0 && V > 0 && s == NAJU_OK) {
                    std::fprintf(stderr, "logits_process without pointers accepted\n");
                    ++failures;
                }
            }

    for (int64_t R : Ts)
        for (int64_t K : Vs)
            for (int64_t G : {(int64_t)0, (int64_t)32, (int64_t)-64, INT64_MIN}) {
                const naju_status_t s = naju_w4_linear(R, K, 5, G, nullptr, nullptr, nullptr,
                                                       nullptr, nullptr, nullptr, nullptr, nullptr);
                if (R > 0 && s == NAJU_OK) {
                    std::fprintf(stderr, "w4_linear without pointers accepted\n");
                    ++failures;
                }
                expect("w4_quantize without pointers",
                       naju_w4_quantize(2, R > 0 ? 3 : -1, G, NAJU_F32, nullptr, nullptr, nullptr,
                                        nullptr, nullptr),
                       G == 32 || R <= 0 ? NAJU_EINVAL : NAJU_EUNSUPPORTED);
            }

    if (failures) return 1;
    std::puts("lm driver: ok");
    return 0;
}
