/*
 * CPU oracle of the residual path: layer norm over the channels, dropout from a counter-based
 * generator with the residual add, and the two in sequence; forward and backward.
 *
 * TEST INFRASTRUCTURE ONLY; shares no code with the CUDA library.  Plain loops in IEEE double,
 * one row (b, t) or one channel at a time, following the definitions:
 *
 *   kept(e):  Philox4x32-10 (Salmon, Moraes, Dror and Shaw, SC 2011), key = seed, counter =
 *             e/8 + 2^64 offset, 16 bits per element; kept when they are >= thr
 *   s = [t < len_b] (res + [kept] mult x)
 *   mean = sum_c s / C, rstd = 1 / sqrt(sum_c (s - mean)^2 / C + eps),
 *   y = [t < len_b] ((s - mean) rstd gamma + beta)
 *   xh = (h - mean) rstd, g = dy gamma, ds = [t < len_b] (dh + rstd (g - sum g / C - xh sum (g xh) / C))
 *   dx = [kept] mult ds, dgamma = sum_{b,t} dy xh, dbeta = sum_{b,t} dy
 */
#include <math.h>
#include <stdint.h>
#include <stddef.h>

static int64_t clamp_len(const int32_t *lengths, int64_t b, int64_t T)
{
    if (lengths == NULL) return T;
    if (lengths[b] < 0) return 0;
    return lengths[b] > T ? T : lengths[b];
}

/* One Philox4x32-10 block: ctr[4] under key[2] into out[4]. */
void oracle_philox4x32(const uint32_t *ctr, const uint32_t *key, uint32_t *out)
{
    uint32_t x[4] = {ctr[0], ctr[1], ctr[2], ctr[3]}, k[2] = {key[0], key[1]};
    for (int round = 0; round < 10; ++round) {
        if (round > 0) {
            k[0] += 0x9E3779B9u;
            k[1] += 0xBB67AE85u;
        }
        const uint64_t p0 = (uint64_t)0xD2511F53u * x[0], p1 = (uint64_t)0xCD9E8D57u * x[2];
        const uint32_t y0 = (uint32_t)(p1 >> 32) ^ x[1] ^ k[0], y1 = (uint32_t)p1;
        const uint32_t y2 = (uint32_t)(p0 >> 32) ^ x[3] ^ k[1], y3 = (uint32_t)p0;
        x[0] = y0; x[1] = y1; x[2] = y2; x[3] = y3;
    }
    for (int i = 0; i < 4; ++i) out[i] = x[i];
}

/* keep[i] = 1 when element first + i is kept, i in [0, n). */
void oracle_dropout_kept(int64_t first, int64_t n, uint64_t seed, uint64_t offset, uint32_t thr, uint8_t *keep)
{
    const uint32_t key[2] = {(uint32_t)seed, (uint32_t)(seed >> 32)};
    #pragma omp parallel for schedule(static)
    for (int64_t k = 0; k < n; ++k) {
        const int64_t e = first + k;
        const uint64_t g = (uint64_t)e / 8;
        const uint32_t ctr[4] = {(uint32_t)g, (uint32_t)(g >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
        uint32_t out[4];
        oracle_philox4x32(ctr, key, out);
        const int i = (int)(e % 8);
        const uint32_t u = i % 2 == 0 ? (out[i / 2] & 0xFFFFu) : (out[i / 2] >> 16);
        keep[k] = u >= thr;
    }
}

/* s = [t < len_b] (res + [kept] mult x); res and keep may be NULL. */
void oracle_dropout_add(const double *x, const double *res, const uint8_t *keep, double mult, const int32_t *lengths,
                        int64_t B, int64_t T, int64_t C, double *s)
{
    #pragma omp parallel for schedule(static)
    for (int64_t r = 0; r < B * T; ++r) {
        const int valid = r % T < clamp_len(lengths, r / T, T);
        for (int64_t c = 0; c < C; ++c) {
            const int64_t e = r * C + c;
            double v = 0.0;
            if (valid) {
                if (keep == NULL || keep[e]) v = mult * x[e];
                if (res != NULL) v += res[e];
            }
            s[e] = v;
        }
    }
}

void oracle_layernorm_fwd(const double *s, const double *gamma, const double *beta, const int32_t *lengths, int64_t B,
                          int64_t T, int64_t C, double eps, double *y, double *mean, double *rstd)
{
    #pragma omp parallel for schedule(static)
    for (int64_t r = 0; r < B * T; ++r) {
        const double *x = s + r * C;
        mean[r] = rstd[r] = 0.0;
        for (int64_t c = 0; c < C; ++c) y[r * C + c] = 0.0;
        if (r % T >= clamp_len(lengths, r / T, T)) continue;
        double m = 0.0, v = 0.0;
        for (int64_t c = 0; c < C; ++c) m += x[c];
        m /= (double)C;
        for (int64_t c = 0; c < C; ++c) v += (x[c] - m) * (x[c] - m);
        mean[r] = m;
        rstd[r] = 1.0 / sqrt(v / (double)C + eps);
        for (int64_t c = 0; c < C; ++c)
            y[r * C + c] = (x[c] - m) * rstd[r] * (gamma ? gamma[c] : 1.0) + (beta ? beta[c] : 0.0);
    }
}

/* ds, dgamma, dbeta; dh may be NULL. */
void oracle_layernorm_bwd(const double *h, const double *dy, const double *dh, const double *gamma,
                          const double *mean, const double *rstd, const int32_t *lengths, int64_t B, int64_t T,
                          int64_t C, double *ds, double *dgamma, double *dbeta)
{
    #pragma omp parallel for schedule(static)
    for (int64_t r = 0; r < B * T; ++r) {
        for (int64_t c = 0; c < C; ++c) ds[r * C + c] = 0.0;
        if (r % T >= clamp_len(lengths, r / T, T)) continue;
        double c1 = 0.0, c2 = 0.0;
        for (int64_t c = 0; c < C; ++c) {
            const double g = dy[r * C + c] * (gamma ? gamma[c] : 1.0);
            c1 += g;
            c2 += g * (h[r * C + c] - mean[r]) * rstd[r];
        }
        c1 /= (double)C;
        c2 /= (double)C;
        for (int64_t c = 0; c < C; ++c) {
            const double g = dy[r * C + c] * (gamma ? gamma[c] : 1.0), xh = (h[r * C + c] - mean[r]) * rstd[r];
            ds[r * C + c] = rstd[r] * (g - c1 - xh * c2) + (dh ? dh[r * C + c] : 0.0);
        }
    }
    #pragma omp parallel for schedule(static)
    for (int64_t c = 0; c < C; ++c) {
        double a = 0.0, b = 0.0;
        for (int64_t r = 0; r < B * T; ++r) {
            if (r % T >= clamp_len(lengths, r / T, T)) continue;
            a += dy[r * C + c] * (h[r * C + c] - mean[r]) * rstd[r];
            b += dy[r * C + c];
        }
        dgamma[c] = a;
        dbeta[c] = b;
    }
}
