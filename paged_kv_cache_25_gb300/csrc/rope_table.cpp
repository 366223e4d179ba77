// Host side of the rotary position embedding: the cos/sin table.
#include <cmath>
#include <cstddef>

#include "../../include/pa.h"

extern "C" int pa_rope_table(float* table, int max_position, int rot_dim, double base)
{
    if (!table || max_position <= 0 || rot_dim <= 0 || rot_dim % 2 != 0 || !(base > 0.0) ||
        !std::isfinite(base))
        return -1;
    const int half = rot_dim / 2;
    for (int p = 0; p < max_position; ++p) {
        float* row = table + static_cast<size_t>(p) * rot_dim;
        for (int i = 0; i < half; ++i) {
            const double a = p * std::pow(base, -2.0 * i / rot_dim);
            row[i] = static_cast<float>(std::cos(a));
            row[half + i] = static_cast<float>(std::sin(a));
        }
    }
    return 0;
}
